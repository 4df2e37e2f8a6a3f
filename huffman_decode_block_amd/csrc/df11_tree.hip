// Attention of drafted tokens over a paged cache (gfx950): a tree or a chain of
// new tokens for each sequence (include/df11_search.h).
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "df11_paged.h"
#include "df11_search.h"

namespace {

using namespace df11p;

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kWaves = 4;
constexpr uint32_t kStep = 32;
constexpr uint32_t kMinChunk = kWaves * kStep;
constexpr uint32_t kMaxChunk = 16384;
constexpr uint32_t kPad = 4;  // floats between rows in LDS: they start in different banks
constexpr float kSlack = 8;   // powers of two that weights may grow to before their reference follows

struct TreeParams {
    Pages k, v;
    const uint16_t *q;
    const int32_t *table, *lens, *counts, *starts;
    const int64_t *mask;
    uint16_t *out;
    float *lse;
    float *part;   // [batch * nodes * q_heads][splits][head_dim]: sums of weighted values
    float *stats;  // [batch * nodes * q_heads][splits][2]: reference (of log2 units) and sum
    uint64_t q_batch, q_node, q_head, mask_batch, mask_node, starts_batch, starts_node, table_stride, n_pages;
    uint32_t batch, nodes, q_heads, kv_heads, group, tiles, splits, page_shift, positions;
    uint32_t units;  // batch * kv_heads * splits
    float scale;     // times log2 e
};

// Bits lo..hi - 1 of 32, both held to [0, 32].
__device__ __forceinline__ uint32_t bits_between(int32_t lo, int32_t hi) {
    const uint32_t l = static_cast<uint32_t>(min(max(lo, 0), 32)), h = static_cast<uint32_t>(min(max(hi, 0), 32));
    const uint64_t below_h = (uint64_t{1} << h) - 1, below_l = (uint64_t{1} << l) - 1;
    return static_cast<uint32_t>(below_h & ~below_l);
}

__device__ __forceinline__ uint32_t pack2h(float a, float b) {
    h2 v;
    v.x = static_cast<_Float16>(a);
    v.y = static_cast<_Float16>(b);
    return __builtin_bit_cast(uint32_t, v);
}

// Two FP16 values from two bytes of E4M3 (exact).
template <bool kHigh>
__device__ __forceinline__ uint32_t half_from_e4m3(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, kHigh));
}

// The parts of a dword's values that are no finite number: all bits of those
// values set, the others clear.
template <bool kE4M3>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    if (kE4M3) {  // NaN: bits 6..0 set
        uint32_t m = w & 0x7F7F7F7Fu;
        m = (m + 0x01010101u) & 0x80808080u;
        return (m >> 7) * 0xFFu;
    }
    uint32_t m = (w & 0x7F807F80u) + 0x00800080u;  // infinities and NaN: bits 14..7 set
    m = (m & 0x80008000u) >> 15;
    return m * 0xFFFFu;
}

// Two values' kinds as BF16 numbers: 1 for infinity, 64 for -infinity, 4096 for
// NaN, 0 for all others; sums of 32 of them tell the kinds apart.
__device__ __forceinline__ uint32_t kind_of(uint32_t bf16) {
    const uint32_t a = bf16 & 0x7FFFu;
    return a < 0x7F80u ? 0u : a > 0x7F80u ? 0x4580u : bf16 & 0x8000u ? 0x4280u : 0x3F80u;
}

template <bool kE4M3, class Row>
__device__ __forceinline__ uint32_t kind2(const Row &row, int j) {
    if (kE4M3) {
        const uint32_t w = row[j / 4] >> (8 * (j & 3));
        return ((w & 0x7Fu) == 0x7Fu ? 0x4580u : 0u) | ((w & 0x7F00u) == 0x7F00u ? 0x45800000u : 0u);
    }
    const uint32_t w = row[kE4M3 ? 0 : j / 2];
    return kind_of(w & 0xFFFFu) | kind_of(w >> 16) << 16;
}

__device__ __forceinline__ float of_counts(float sum) {
    const uint32_t n = static_cast<uint32_t>(sum), plus = n & 63u, minus = n >> 6 & 63u;
    return n >> 12 || (plus && minus) ? NAN : plus ? INFINITY : minus ? -INFINITY : 0.0f;
}

constexpr int waves_for(int dim, int tiles) { return dim * tiles <= 64 ? 3 : dim * tiles <= 256 && dim < 256 ? 2 : 1; }

template <int kDim, bool kE4M3, int kTiles>
__global__ void __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(waves_for(kDim, kTiles))))
tree_kernel(TreeParams p) {
    constexpr int kPiece = kDim / 16;              // values of a V row in a lane; tiles of out^T
    constexpr int kKChunks = kDim / 32;            // matrix instructions over d
    constexpr int kKLoads = kE4M3 ? kDim / 64 : kKChunks;  // 16-byte loads of a K row in a lane
    constexpr int kVWords = kPiece * (kE4M3 ? 1 : 2) / 4;  // dwords of a V piece
    constexpr uint32_t kRows = 16 * kTiles;
    __shared__ int32_t s_page[kMaxChunk / kMinPage + 1];
    __shared__ float s_stat[kWaves][2][16];
    __shared__ __attribute__((aligned(16))) float s_out[kWaves][16][kDim + kPad];

    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // workgroups go round the 8 XCDs: those of one chunk's tiles, which read the
    // same keys and values, stay on one
    const uint32_t turn = blockIdx.x / (8 * p.tiles), in = blockIdx.x - turn * 8 * p.tiles;
    const uint32_t tile = in / 8;
    uint32_t unit = turn * 8 + (in & 7u);
    if (unit >= p.units) return;
    const uint32_t h = unit % p.kv_heads;
    unit /= p.kv_heads;
    const uint32_t b = unit % p.batch, split = unit / p.batch;

    // this tile's rows: row n is node n / group, head n % group
    const uint32_t row0 = tile * kRows, rows = min(kRows, p.nodes * p.group - row0);
    const int32_t count = min(max(p.counts ? p.counts[b] : INT32_MAX, 0), static_cast<int32_t>(p.nodes));
    const int32_t len = static_cast<int32_t>(min(static_cast<uint32_t>(max(p.lens[b], 0)), p.positions));
    const int32_t node_first = static_cast<int32_t>(row0 / p.group), node_last = static_cast<int32_t>((row0 + rows - 1) / p.group);
    int32_t node[kTiles], start[kTiles];
    bool have[kTiles];
    int32_t lo = len, lo_max = 0;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const uint32_t n = row0 + 16 * t + r;
        node[t] = static_cast<int32_t>(min(n, p.nodes * p.group - 1) / p.group);
        have[t] = 16 * t + r < rows && node[t] < count;
        start[t] = 0;
        if (p.starts) start[t] = min(max(p.starts[b * p.starts_batch + static_cast<uint32_t>(node[t]) * p.starts_node], 0), len);
        lo = have[t] ? min(lo, start[t]) : lo;
        lo_max = have[t] ? max(lo_max, start[t]) : lo_max;
    }
    if (p.starts) {
#pragma unroll
        for (int i = 1; i < 16; i <<= 1) {
            lo = min(lo, __shfl_xor(lo, i));
            lo_max = max(lo_max, __shfl_xor(lo_max, i));
        }
        lo = __builtin_amdgcn_readfirstlane(lo);
        lo_max = __builtin_amdgcn_readfirstlane(lo_max);
    } else {
        lo = lo_max = 0;
    }
    // the positions that any of these rows reads, and those that all read
    const int32_t reach = min(count, p.mask ? count : node_last + 1);
    const int32_t hi = node_first < count ? static_cast<int32_t>(min(static_cast<uint32_t>(len) + reach, p.positions)) : 0;
    const int32_t all_hi = p.mask ? len : min(len + min(node_first + 1, count), hi);
    const int32_t base = lo & ~static_cast<int32_t>(kStep - 1);
    const uint32_t steps = hi > base ? (hi - base + kStep - 1) / kStep : 0;
    const bool single = p.splits == 1;
    const uint32_t chunks = min(p.splits, (steps + kWaves - 1) / kWaves);
    const auto out_row = [&](uint32_t i) {  // of the tile's row i
        const uint32_t n = row0 + i, nd = n / p.group;
        return (uint64_t{b} * p.nodes + nd) * p.q_heads + h * p.group + (n - nd * p.group);
    };
    if (!single && split >= chunks) {  // nothing here: the join gives it no weight
        for (uint32_t i = threadIdx.x; i < rows; i += 64 * kWaves) {
            float *to = p.stats + 2 * (out_row(i) * p.splits + split);
            to[0] = -INFINITY;
            to[1] = 0;
        }
        return;
    }
    const uint32_t parts = max(chunks, 1u), each = steps / parts, more = steps - each * parts;
    const int32_t c0 = base + static_cast<int32_t>((split * each + min(split, more)) * kStep);
    const int32_t c1 = max(c0, min(c0 + static_cast<int32_t>((each + (split < more)) * kStep), hi));

    // the chunk's pages; -1 masks
    const uint32_t first = static_cast<uint32_t>(c0) >> p.page_shift;
    const uint32_t n_pages = c1 > c0 ? (static_cast<uint32_t>(c1 - 1) >> p.page_shift) - first + 1 : 0;
    const int32_t *table = p.table + b * p.table_stride + first;
    int32_t masked_pages = 0;
    for (uint32_t i = threadIdx.x; i < n_pages; i += 64 * kWaves) {
        const int32_t e = table[i];
        const bool ok = e >= 0 && static_cast<uint64_t>(e) < p.n_pages;
        s_page[i] = ok ? e : -1;
        masked_pages |= !ok;
    }

    // Q^T: row r of each tile, d in the order in which K's loads give them.  A
    // negative scale turns q around, so that the largest product is the largest score.
    const float signed_scale = kE4M3 ? p.scale * p.k.scale[h] : p.scale;
    const float scale = fabsf(signed_scale);
    const uint32_t turned = signed_scale < 0 ? 0x80008000u : 0;
    bf8 qf[kTiles][kKChunks];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const uint32_t n = min(row0 + 16 * t + r, p.nodes * p.group - 1);
        const uint16_t *qp = p.q + b * p.q_batch + static_cast<uint32_t>(node[t]) * p.q_node +
                             (h * p.group + (n - static_cast<uint32_t>(node[t]) * p.group)) * p.q_head;
#pragma unroll
        for (int i = 0; i < kKChunks; ++i) {
            const uint32_t d = kE4M3 ? 64 * (i / 2) + 16 * q + 8 * (i & 1) : 32 * i + 8 * q;
            v4u w = have[t] ? load8(qp + d) : v4u{0, 0, 0, 0};
            w ^= turned;
            qf[t][i] = __builtin_bit_cast(bf8, w);
        }
    }
    const uint8_t *kb = p.k.base + h * p.k.head, *vb = p.v.base + h * p.v.head;
    const uint32_t in_page = (1u << p.page_shift) - 1;
    const bool holes = __syncthreads_or(masked_pages);  // and the pages are there

    // K rows of a step: lane r has position r of each half
    v4u kr[2][kKLoads];
    auto load_k = [&](int32_t p0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t pos = static_cast<uint32_t>(min(p0 + 16 * t + static_cast<int32_t>(r), c1 - 1));
            const int32_t page = max(s_page[(pos >> p.page_shift) - first], 0);
            const uint8_t *row = kb + static_cast<uint64_t>(page) * p.k.page + uint64_t{pos & in_page} * p.k.row + 16 * q;
#pragma unroll
            for (int i = 0; i < kKLoads; ++i) kr[t][i] = *reinterpret_cast<const v4u *>(row + 64 * i);
        }
    };
    // V rows of a step: positions 4 q + 0..3 of each half (of one page: pages
    // hold multiples of 8)
    typedef uint32_t VRow __attribute__((ext_vector_type(kVWords)));
    typedef VRow VRowInMemory __attribute__((aligned(4)));
    VRow vr[8];
    auto load_v = [&](int32_t p0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int32_t pos0 = p0 + 16 * t + 4 * static_cast<int32_t>(q);
            const int32_t page = s_page[(static_cast<uint32_t>(min(pos0, c1 - 1)) >> p.page_shift) - first];
            const uint8_t *at_page = vb + static_cast<uint64_t>(max(page, 0)) * p.v.page + r * (kVWords * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t at = static_cast<uint32_t>(min(pos0 + i, c1 - 1));
                vr[4 * t + i] = *reinterpret_cast<const VRowInMemory *>(at_page + uint64_t{at & in_page} * p.v.row);
            }
        }
    };
    // Which of a lane's eight positions lie in the chunk, past every start and in pages of the cache.
    auto positions_there = [&](int32_t p0) {
        uint32_t there = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int32_t pos0 = p0 + 16 * t + 4 * static_cast<int32_t>(q);
            const bool page = s_page[(static_cast<uint32_t>(min(pos0, c1 - 1)) >> p.page_shift) - first] >= 0;
            there |= page ? (bits_between(lo - pos0, c1 - pos0) & 15u) << (4 * t) : 0u;
        }
        return there;
    };
    // Which of them row r of a tile reads.
    auto positions_read = [&](int t, int32_t p0) {
        uint32_t live = bits_between(start[t] - p0, len - p0);
        const int32_t a0 = p0 - len;  // the node at p0
        if (a0 + static_cast<int32_t>(kStep) > 0) {
            if (!p.mask) {
                live |= bits_between(-a0, min(node[t] + 1, count) - a0);
            } else if (a0 < count) {
                const int64_t *words = p.mask + b * p.mask_batch + static_cast<uint32_t>(node[t]) * p.mask_node;
                const uint32_t from = static_cast<uint32_t>(max(a0, 0));
                const uint32_t w = from / 64, shift = from % 64;
                uint64_t m = static_cast<uint64_t>(words[w]) >> shift;
                if (shift > 32 && 64 * (w + 1) < p.nodes) m |= static_cast<uint64_t>(words[w + 1]) << (64 - shift);
                live |= static_cast<uint32_t>(a0 < 0 ? m << -a0 : m) & bits_between(-a0, count - a0);
            }
        }
        return ((live >> (4 * q)) & 15u) | (((live >> (16 + 4 * q)) & 15u) << 4);
    };

    float ref[kTiles], l[kTiles];  // reference of a row's weights in log2 units, their sum over this lane's positions
    f4 acc[kTiles][kPiece] = {};
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        ref[t] = -INFINITY;
        l[t] = 0;
    }

    auto step = [&](int32_t p0, int32_t next, auto masked_) {
        constexpr bool kMasked = decltype(masked_)::value;
        f4 s[kTiles][2] = {};
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < kKChunks; ++i) {
                v4u kw;
                if (kE4M3)
                    kw = i & 1 ? from_e4m3x8(kr[u][i / 2].z, kr[u][i / 2].w) : from_e4m3x8(kr[u][i / 2].x, kr[u][i / 2].y);
                else
                    kw = kr[u][kE4M3 ? 0 : i];
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
                    s[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, kw), qf[t][i], s[t][u], 0, 0, 0);
            }
        load_k(next);

        uint32_t there = 0xFF, odd = 0;  // odd: some value of V is no finite number
        if (kMasked) {
            there = positions_there(p0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                vr[i] = there >> i & 1u ? vr[i] : VRow(0);
#pragma unroll
                for (int w = 0; w < kVWords; ++w) {
                    const uint32_t n = not_finite<kE4M3>(vr[i][w]);
                    odd |= n;
                    vr[i][w] &= ~n;
                }
            }
            odd = __any(odd != 0);
        }
        v4u high[kTiles], low[kTiles];  // the weights as the product takes them
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            uint32_t live = 0xFF;
            if (kMasked) {
                live = positions_read(t, p0) & there;
#pragma unroll
                for (int i = 0; i < 8; ++i) s[t][i / 4][i & 3] = live >> i & 1u ? s[t][i / 4][i & 3] : -INFINITY;
            }
            float top = s[t][0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, s[t][i / 4][i & 3]);
            // the reference follows a maximum that has left it behind
            const bool behind = top > -INFINITY && !(top * scale <= ref[t] + kSlack);
            if (__any(behind)) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float to = top > -INFINITY ? fmaxf(ref[t], top * scale) : ref[t];
                const float fade = to == ref[t] ? 1.0f : exp2_(ref[t] - to);
                ref[t] = to;
                l[t] *= fade;
#pragma unroll
                for (int j = 0; j < kPiece; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[t][j][c] *= fade;
            }
            const float from = ref[t] == -INFINITY ? 0.0f : ref[t];
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = exp2_(fmaf(s[t][i / 4][i & 3], scale, -from));
                if (kMasked) w[i] = live >> i & 1u ? w[i] : 0.0f;
                l[t] += w[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (kE4M3) {
                    high[t][i] = pack2h(w[2 * i], w[2 * i + 1]);
                } else {
                    high[t][i] = cut2(w[2 * i], w[2 * i + 1]);
                    low[t][i] = pack2(w[2 * i] - __builtin_bit_cast(float, high[t][i] << 16),
                                      w[2 * i + 1] - __builtin_bit_cast(float, high[t][i] & 0xFFFF0000u));
                    if (!kMasked) low[t][i] = at_least2(low[t][i], kLeastPart);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kPiece; j += 2) {
            // values j and j + 1 of the eight rows
            uint32_t pair[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (kE4M3)
                    pair[i] = j & 2 ? half_from_e4m3<true>(vr[i][j / 4]) : half_from_e4m3<false>(vr[i][j / 4]);
                else
                    pair[i] = vr[i][kE4M3 ? 0 : j / 2];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t sel = e ? 0x07060302u : 0x05040100u;
                const v4u a = {__builtin_amdgcn_perm(pair[1], pair[0], sel), __builtin_amdgcn_perm(pair[3], pair[2], sel),
                               __builtin_amdgcn_perm(pair[5], pair[4], sel), __builtin_amdgcn_perm(pair[7], pair[6], sel)};
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    f4 o = acc[t][j + e];
                    if (kE4M3) {
                        o = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, high[t]), o, 0, 0, 0);
                    } else {
                        o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, high[t]), o, 0, 0, 0);
                        o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, low[t]), o, 0, 0, 0);
                    }
                    acc[t][j + e] = o;
                }
            }
        }
        if (kMasked && odd) {
            // What is no finite number was left out above, as 0 times it would reach
            // rows that do not read it.  A product of ones counts for each row how many
            // of those that it reads are infinities of either sign or NaN.
            load_v(p0);
            uint32_t ones[kTiles][4];
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const uint32_t live = positions_read(t, p0) & there;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ones[t][i] = (live >> (2 * i) & 1u ? 0x3F80u : 0u) | (live >> (2 * i + 1) & 1u ? 0x3F800000u : 0u);
            }
#pragma unroll
            for (int j = 0; j < kPiece; j += 2) {
                uint32_t pair[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) pair[i] = there >> i & 1u ? kind2<kE4M3>(vr[i], j) : 0u;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t sel = e ? 0x07060302u : 0x05040100u;
                    const bf8 a = __builtin_bit_cast(
                        bf8, v4u{__builtin_amdgcn_perm(pair[1], pair[0], sel), __builtin_amdgcn_perm(pair[3], pair[2], sel),
                                 __builtin_amdgcn_perm(pair[5], pair[4], sel), __builtin_amdgcn_perm(pair[7], pair[6], sel)});
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) {
                        const bf8 w = __builtin_bit_cast(bf8, v4u{ones[t][0], ones[t][1], ones[t][2], ones[t][3]});
                        const f4 n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, w, f4{}, 0, 0, 0);
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[t][j + e][c] += of_counts(n[c]);
                    }
                }
            }
        }
        load_v(next);
    };
    const auto masked_at = [&](int32_t p0) { return holes || p0 < lo_max || p0 + static_cast<int32_t>(kStep) > min(all_hi, c1); };
    int32_t p0 = c0 + static_cast<int32_t>(wave * kStep);
    if (p0 < c1) {
        load_k(p0);
        load_v(p0);
        // the last step loads its chunk's last row in vain
        for (; p0 < c1; p0 += kWaves * kStep) {
            if (masked_at(p0))
                step(p0, p0 + kWaves * kStep, std::true_type());
            else
                step(p0, p0 + kWaves * kStep, std::false_type());
        }
    }

    // join the waves, a tile at a time
    const float v_scale = kE4M3 ? p.v.scale[h] : 1.0f;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        if (16u * t >= rows) break;
        float sum = l[t];
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (t) __syncthreads();  // the last tile has been read
        if (q == 0) {
            s_stat[wave][0][r] = ref[t];
            s_stat[wave][1][r] = sum;
        }
        // acc[j][c]: d = (4 q + c) * kPiece + j
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < kPiece; j += 4)
                *reinterpret_cast<f4 *>(&s_out[wave][r][(4 * q + c) * kPiece + j]) =
                    f4{acc[t][j][c], acc[t][j + 1][c], acc[t][j + 2][c], acc[t][j + 3][c]};
        __syncthreads();
        constexpr uint32_t kQuads = kDim / 4;
        for (uint32_t i = threadIdx.x; i < min(16u, rows - 16 * t) * kQuads; i += 64 * kWaves) {
            const uint32_t g = i / kQuads, d = i % kQuads * 4;
            const bool there = static_cast<int32_t>((row0 + 16 * t + g) / p.group) < count;
            float top = -INFINITY;
#pragma unroll
            for (uint32_t k = 0; k < kWaves; ++k) top = fmaxf(top, s_stat[k][0][g]);
            if (!there) top = -INFINITY;
            const float from = top == -INFINITY ? 0.0f : top;
            float total = 0;
            f4 o = {};
#pragma unroll
            for (uint32_t k = 0; k < kWaves; ++k) {
                const float f = exp2_(s_stat[k][0][g] - from);
                total += s_stat[k][1][g] * f;
                o += *reinterpret_cast<const f4 *>(&s_out[k][g][d]) * f;
            }
            if (!there) {
                total = 0;
                o = f4{};
            }
            o *= v_scale;
            const uint64_t row = out_row(16 * t + g);
            if (single) {
                if (total == 0) o = f4{};
                const float inv = total == 0 ? 0.0f : 1.0f / total;
                v2u to;
                to.x = pack2(o[0] * inv, o[1] * inv);
                to.y = pack2(o[2] * inv, o[3] * inv);
                *reinterpret_cast<v2u *>(p.out + row * kDim + d) = to;
                if (d == 0 && p.lse) p.lse[row] = (from + __builtin_amdgcn_logf(total)) * kLn2;
            } else {
                const uint64_t at = row * p.splits + split;
                *reinterpret_cast<f4 *>(p.part + at * kDim + d) = o;
                if (d == 0) {
                    p.stats[2 * at] = top;
                    p.stats[2 * at + 1] = total;
                }
            }
        }
    }
}

// Joins the chunks: kDim / 4 lanes for a row, four values each.
constexpr uint32_t kJoinThreads = 256;

template <int kDim>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(TreeParams p, uint64_t rows) {
    constexpr uint32_t kQuads = kDim / 4;
    const uint64_t row = uint64_t{blockIdx.x} * (kJoinThreads / kQuads) + threadIdx.x / kQuads;
    const uint32_t d = threadIdx.x % kQuads;
    if (row >= rows) return;
    const v2f *stats = reinterpret_cast<const v2f *>(p.stats) + row * p.splits;
    const f4 *part = reinterpret_cast<const f4 *>(p.part + row * p.splits * kDim) + d;
    float top = -INFINITY;
    for (uint32_t i = 0; i < p.splits; ++i) top = fmaxf(top, stats[i].x);
    const float from = top == -INFINITY ? 0.0f : top;
    float total = 0;
    f4 o = {};
    for (uint32_t i = 0; i < p.splits; ++i) {
        const v2f s = stats[i];
        if (s.x == -INFINITY && s.y == 0) continue;  // its values are not written
        const float f = exp2_(s.x - from);
        total += s.y * f;
        o += part[uint64_t{i} * kQuads] * f;
    }
    if (total == 0) o = f4{};
    const float inv = total == 0 ? 0.0f : 1.0f / total;
    v2u to;
    to.x = pack2(o[0] * inv, o[1] * inv);
    to.y = pack2(o[2] * inv, o[3] * inv);
    *reinterpret_cast<v2u *>(p.out + row * kDim + 4 * d) = to;
    if (d == 0 && p.lse) p.lse[row] = (from + __builtin_amdgcn_logf(total)) * kLn2;
}

// ---- Host ------------------------------------------------------------------

struct Shape {
    uint32_t row_tiles;  // of 16 rows in a workgroup
    uint32_t tiles, splits;
};

constexpr uint64_t kWantGroups = 2 * kComputeUnits;

Shape shape_of(uint64_t batch, uint64_t nodes, uint32_t group, uint32_t kv_heads, uint32_t dim, uint64_t positions) {
    const uint64_t rows = nodes * group;
    Shape s;
    s.row_tiles = rows <= 16 ? 1 : rows <= 32 || dim == 256 ? 2 : 4;
    s.tiles = static_cast<uint32_t>((rows + 16 * s.row_tiles - 1) / (16 * s.row_tiles));
    const uint64_t units = batch * kv_heads * s.tiles;
    const uint64_t want = (kWantGroups + units - 1) / std::max<uint64_t>(units, 1);
    const uint64_t most = (positions + kMinChunk - 1) / kMinChunk, least = (positions + kMaxChunk - 1) / kMaxChunk;
    s.splits = static_cast<uint32_t>(positions <= 2 * kMinChunk ? 1 : std::max(std::min(want, most), least));
    return s;
}

bool sizes_ok(uint64_t batch, uint64_t nodes, uint32_t q_heads, uint32_t kv_heads, uint32_t page_size, uint64_t width) {
    return batch <= (1u << 24) && nodes <= (1u << 20) && kv_heads > 0 && kv_heads <= 65536 && q_heads > 0 && q_heads <= (1u << 20) &&
           q_heads % kv_heads == 0 && width > 0 && width < (1u << 30) / page_size;
}

uint64_t workgroups(uint64_t batch, uint32_t kv_heads, const Shape &s) {
    return (batch * kv_heads * s.splits + 7) / 8 * 8 * s.tiles;
}

// Whether the kernels' work items fit a launch, which holds fewer than 2^32.
bool launchable(uint64_t batch, uint64_t nodes, uint32_t q_heads, uint32_t kv_heads, const Shape &s) {
    return batch * kv_heads * s.splits < (uint64_t{1} << 32) && workgroups(batch, kv_heads, s) < (1u << 24) &&
           nodes * q_heads < (uint64_t{1} << 31) && batch * nodes * q_heads < (uint64_t{1} << 31) / 64 * 16;
}

uint64_t workspace_of(uint64_t batch, uint64_t nodes, uint32_t q_heads, uint32_t dim, const Shape &s) {
    return s.splits <= 1 ? 0 : batch * nodes * q_heads * s.splits * (dim + 2) * sizeof(float);
}

template <int kDim>
auto kernel_of(bool e4m3, uint32_t row_tiles) {
    if constexpr (kDim < 256)
        if (row_tiles == 4) return e4m3 ? tree_kernel<kDim, true, 4> : tree_kernel<kDim, false, 4>;
    if (row_tiles == 1) return e4m3 ? tree_kernel<kDim, true, 1> : tree_kernel<kDim, false, 1>;
    return e4m3 ? tree_kernel<kDim, true, 2> : tree_kernel<kDim, false, 2>;
}

df11_status tree_attention(const df11_paged_cache *c, const df11_tree *t, const int32_t *table, uint64_t table_stride,
                           uint64_t width, const int32_t *lens, uint16_t *out, float *lse, void *workspace,
                           uint64_t workspace_bytes, void *hip_stream) {
    const df11_status rc = check_cache(c);
    if (rc != DF11_OK) return rc;
    if (!t || !sizes_ok(t->batch, t->nodes, t->q_heads, c->kv_heads, c->page_size, width)) return DF11_E_INVALID_ARG;
    for (uint64_t s : {t->q_batch_stride, t->q_node_stride, t->q_head_stride, t->mask_batch_stride, t->mask_node_stride,
                       t->starts_batch_stride, t->starts_node_stride, table_stride})
        if (s > kMaxStride) return DF11_E_INVALID_ARG;
    if (table_stride < width || span(t->batch, table_stride) >= kMaxExtent ||
        span(t->batch, t->q_batch_stride) + span(t->nodes, t->q_node_stride) + span(t->q_heads, t->q_head_stride) >= kMaxExtent ||
        span(t->batch, t->starts_batch_stride) + span(t->nodes, t->starts_node_stride) >= kMaxExtent ||
        span(t->batch, t->mask_batch_stride) + span(t->nodes, t->mask_node_stride) >= kMaxExtent)
        return DF11_E_INVALID_ARG;
    if (t->batch == 0 || t->nodes == 0) return DF11_OK;
    if (t->mask && t->nodes > 1 && t->mask_node_stride < (t->nodes + 63) / 64) return DF11_E_INVALID_ARG;
    const auto low = [](const void *p) { return reinterpret_cast<uintptr_t>(p); };
    if (!t->q || !table || !lens || !out || (low(t->q) & 1u) || !aligned16(out) || (low(t->mask) & 7u) ||
        ((low(table) | low(lens) | low(t->counts) | low(t->starts) | low(lse)) & 3u) || !aligned16(workspace))
        return DF11_E_INVALID_ARG;
    TreeParams p;
    p.k = k_of(c);
    p.v = v_of(c);
    p.q = t->q;
    p.table = table;
    p.lens = lens;
    p.counts = t->counts;
    p.starts = t->starts;
    p.mask = t->mask;
    p.out = out;
    p.lse = lse;
    p.q_batch = t->q_batch_stride;
    p.q_node = t->q_node_stride;
    p.q_head = t->q_head_stride;
    p.mask_batch = t->mask_batch_stride;
    p.mask_node = t->mask_node_stride;
    p.starts_batch = t->starts_batch_stride;
    p.starts_node = t->starts_node_stride;
    p.table_stride = table_stride;
    p.n_pages = c->n_pages;
    p.batch = static_cast<uint32_t>(t->batch);
    p.nodes = static_cast<uint32_t>(t->nodes);
    p.q_heads = t->q_heads;
    p.kv_heads = c->kv_heads;
    p.group = t->q_heads / c->kv_heads;
    p.page_shift = log2_of(c->page_size);
    p.positions = static_cast<uint32_t>(width * c->page_size);
    p.scale = t->scale * kLog2e;
    const Shape s = shape_of(t->batch, t->nodes, p.group, p.kv_heads, c->head_dim, p.positions);
    if (!launchable(t->batch, t->nodes, t->q_heads, c->kv_heads, s)) return DF11_E_INVALID_ARG;
    p.tiles = s.tiles;
    p.splits = s.splits;
    p.units = static_cast<uint32_t>(t->batch * c->kv_heads * s.splits);
    if (workspace_bytes < workspace_of(t->batch, t->nodes, t->q_heads, c->head_dim, s)) return DF11_E_BUFFER_TOO_SMALL;
    if (s.splits > 1 && !workspace) return DF11_E_INVALID_ARG;
    const uint64_t rows = t->batch * t->nodes * t->q_heads;
    p.part = static_cast<float *>(workspace);
    p.stats = s.splits > 1 ? p.part + rows * s.splits * c->head_dim : nullptr;
    const bool e4m3 = c->dtype == DF11_CACHE_E4M3;
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    auto fn = c->head_dim == 64    ? kernel_of<64>(e4m3, s.row_tiles)
              : c->head_dim == 128 ? kernel_of<128>(e4m3, s.row_tiles)
                                   : kernel_of<256>(e4m3, s.row_tiles);
    hipError_t err = launch(fn, static_cast<uint32_t>(workgroups(t->batch, c->kv_heads, s)), 64 * kWaves, 0, st, p);
    if (err == hipSuccess && s.splits > 1) {
        const uint64_t per = kJoinThreads / (c->head_dim / 4);
        err = launch(c->head_dim == 64    ? tree_join_kernel<64>
                     : c->head_dim == 128 ? tree_join_kernel<128>
                                          : tree_join_kernel<256>,
                     static_cast<uint32_t>((rows + per - 1) / per), kJoinThreads, 0, st, p, rows);
    }
    return launched(err);
}

}  // namespace

extern "C" uint64_t df11_paged_tree_attention_workspace_bytes(uint64_t batch, uint64_t nodes, uint32_t q_heads,
                                                              uint32_t kv_heads, uint32_t head_dim, uint32_t page_size,
                                                              uint64_t table_width) {
    if (!dim_ok(head_dim) || !page_ok(page_size) || !sizes_ok(batch, nodes, q_heads, kv_heads, page_size, table_width)) return 0;
    const Shape s = shape_of(batch, nodes, q_heads / kv_heads, kv_heads, head_dim, table_width * page_size);
    return launchable(batch, nodes, q_heads, kv_heads, s) ? workspace_of(batch, nodes, q_heads, head_dim, s) : 0;
}

extern "C" df11_status df11_paged_tree_attention(const df11_paged_cache *cache, const df11_tree *tree,
                                                 const int32_t *page_table, uint64_t table_stride, uint64_t table_width,
                                                 const int32_t *lens, uint16_t *out, float *lse, void *workspace,
                                                 uint64_t workspace_bytes, void *hip_stream) {
    return df11i::guarded([&] {
        return tree_attention(cache, tree, page_table, table_stride, table_width, lens, out, lse, workspace, workspace_bytes,
                              hip_stream);
    });
}
