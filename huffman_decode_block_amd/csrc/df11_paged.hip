// Paged key-value cache (gfx950): writing new tokens into it and the
// attention of one new token for each sequence (include/df11_step.h).
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "df11_paged.h"

namespace {

using namespace df11p;

// ---- Append ----------------------------------------------------------------
// A lane moves 8 values of K and the same 8 of V.  Bound by the launch for the
// tokens of a step (32 tokens of 8 heads of 128: 2.7 us, the shortest a kernel
// takes here), by HBM for a prompt (8,192 tokens into BF16 pages: 67 MB in 12.8
// us, 5.2 TB/s).  Into E4M3 pages, a tenth of the tokens padding, 46 MB take
// 13.0 us, 3.5 TB/s (11.4 for a call among others, whose start the one before
// hides): not by HBM alone; the conversion's arithmetic and stores half as wide
// are what differs.

struct AppendParams {
    Pages k, v;
    const uint16_t *ks, *vs;
    uint64_t k_token, k_head, v_token, v_head;  // source strides, elements
    const int64_t *slots;
    uint64_t lanes;  // tokens * per_token
    uint64_t n_slots;
    uint32_t per_token, dim_shift, page_shift;  // kv_heads * head_dim / 8; head_dim / 8 = 1 << dim_shift
};

// x / scale for the eight values of a lane, rounded as a division: with r the
// rounded reciprocal and q = x r, q + (x - q scale) r is the rounded quotient
// (Markstein) as long as nothing over- or underflows; quotients of 1024 and
// more are past E4M3 and keep q, and a scale without a normal reciprocal takes
// the division itself.  E4M3's conversion turns magnitudes over 448 into NaN,
// so they are held to 448 before it; NaN is let through.
struct Scale {
    float s, r;
    bool plain;
};

__device__ __forceinline__ Scale scale_of(float s) {
    const float r = 1.0f / s, a = fabsf(r);
    return Scale{s, r, !(a >= 0x1p-100f && a <= 0x1p100f)};
}

__device__ __forceinline__ float to_e4m3_range(uint32_t bits, const Scale &s) {
    const float x = __builtin_bit_cast(float, bits);
    float v;
    if (s.plain) {
        v = x / s.s;
    } else {
        const float q = x * s.r;
        // the correction turns -0 into 0
        v = copysignf(fabsf(q) < 1024.0f ? fmaf(fmaf(-q, s.s, x), s.r, q) : q, q);
    }
    return v != v ? v : fminf(fmaxf(v, -448.0f), 448.0f);
}

__device__ __forceinline__ v2u e4m3x8(v4u x, float scale) {
    const Scale s = scale_of(scale);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int r = 0;
        r = __builtin_amdgcn_cvt_pk_fp8_f32(to_e4m3_range(w[2 * i] << 16, s), to_e4m3_range(w[2 * i] & 0xFFFF0000u, s), r,
                                            false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(to_e4m3_range(w[2 * i + 1] << 16, s),
                                            to_e4m3_range(w[2 * i + 1] & 0xFFFF0000u, s), r, true);
        o[i] = static_cast<uint32_t>(r);
    }
    return v2u{o[0], o[1]};
}

template <bool kE4M3>
__global__ void __launch_bounds__(256) append_kernel(AppendParams p) {
    const uint32_t per_head = 1u << p.dim_shift;
    for (uint64_t base = uint64_t{blockIdx.x} * 256; base < p.lanes; base += uint64_t{gridDim.x} * 256) {
        if (base + threadIdx.x >= p.lanes) break;
        const uint64_t t0 = base / p.per_token;  // uniform
        const uint32_t local = static_cast<uint32_t>(base - t0 * p.per_token) + threadIdx.x;
        const uint32_t down = local / p.per_token, in = local - down * p.per_token;
        const uint64_t t = t0 + down;
        const uint32_t d = in & (per_head - 1), h = in >> p.dim_shift;
        const int64_t slot = p.slots[t];
        if (slot < 0 || static_cast<uint64_t>(slot) >= p.n_slots) continue;
        const v4u kv = load8(p.ks + t * p.k_token + h * p.k_head + 8 * d);
        const v4u vv = load8(p.vs + t * p.v_token + h * p.v_head + 8 * d);
        const uint64_t page = static_cast<uint64_t>(slot) >> p.page_shift;
        const uint64_t row = static_cast<uint64_t>(slot) & ((uint64_t{1} << p.page_shift) - 1);
        uint8_t *ko = p.k.base + page * p.k.page + h * p.k.head + row * p.k.row;
        uint8_t *vo = p.v.base + page * p.v.page + h * p.v.head + row * p.v.row;
        if (kE4M3) {
            *reinterpret_cast<v2u *>(ko + 8 * d) = e4m3x8(kv, p.k.scale[h]);
            *reinterpret_cast<v2u *>(vo + 8 * d) = e4m3x8(vv, p.v.scale[h]);
        } else {
            *reinterpret_cast<v4u *>(ko + 16 * d) = kv;
            *reinterpret_cast<v4u *>(vo + 16 * d) = vv;
        }
    }
}

// ---- Attention of one token ------------------------------------------------
// A sequence's positions are cut into chunks of steps of 32 positions, by the
// lengths as the device finds them; a workgroup takes one chunk of one cache
// head for up to 16 of its query heads, its four waves the chunk's steps in
// turn.  Each wave keeps the running maximum, sum and weighted values of what it
// has seen, the waves join in LDS, and a second kernel joins the chunks.  The
// host knows the page table's width and not the lengths, so it chooses one of
// three ways to share the work (Order), and the device fits it to the lengths:
//   kAsGiven   every sequence is cut into up to `splits` chunks of 128 or more
//   kByLength  one chunk each; compute units get long and short sequences in turn
//   kEvenly    chunks of one length for all sequences, long ones have more of them
//
// Products are matrix instructions of 16 x 16 x 32 in this orientation:
//   scores^T [position, head] = K [position, d] Q^T [d, head]
//   out^T    [d, head]        = V^T [d, position] W^T [position, head]
// A lane (r = lane % 16, q = lane / 16) receives the scores of head r at
// positions 4 q + 0..3 of each half of the step, and the second product wants
// of it, for head r, eight positions of the lane's choice, as long as V^T uses
// the same ones: the weights stay in their lane.  For V^T the lane needs, for
// each of its d, those eight positions: it loads a piece of head_dim / 16
// values of each of the eight rows and transposes inside its own registers
// (byte permutes), d = r * head_dim / 16 + j being the row r of the j-th tile.
// No operand goes through LDS.
//
// The weights exp(s - m) lie in [0, 1]; one BF16 number would add an error as
// large as the output's own rounding, so they are given as two, high part and
// remainder.  A BF16 V may hold infinities, which a weight keeps only if neither
// part is zero or negative: there the high part is cut off, not rounded, which
// leaves a remainder that is not negative, and the remainder is at least 2^-126
// (both parts together are off by up to 2^-16 of the weight, by 2^-17 with a
// rounded high part, which E4M3's V, without infinities, gets; no time was
// lost by it).  The matrix unit has time for two products: the kernel is bound
// by reading K and V, each once.  At 8 sequences of 32,768 positions, 8 cache
// heads of 128 and 64 query heads: BF16 1.07 GB in 184 us, 5.8 TB/s; E4M3 537 MB
// in 94, 5.7 TB/s.  Where there is less to read the start and the end count: one
// sequence of 8,192 takes 9.2 us and its join 3.8 (33.5 MB would take 5.8 at the
// former rate), 64 ragged ones up to 1,024 positions 27 us for 134 MB.

constexpr uint32_t kWaves = 4;
constexpr uint32_t kStep = 32;
constexpr uint32_t kMinChunk = kWaves * kStep;
constexpr uint32_t kMaxChunk = 4096;
constexpr uint32_t kHeadTile = 16;
constexpr uint32_t kLaneSequences = 256;  // sequences that a wave's lanes can hold
constexpr uint32_t kClassBits = 8;

enum Order { kAsGiven, kByLength, kEvenly };  // order_of has the rule and its figures
constexpr uint32_t kPad = 4;  // floats between a head's values in LDS: the heads start in different banks

struct AttnParams {
    Pages k, v;
    const uint16_t *q;
    const int32_t *table, *lens, *starts;
    uint16_t *out;
    float *lse;
    float *part;   // [batch * q_heads][splits][head_dim]: sums of weighted values
    float *stats;  // [batch * q_heads][splits][2]: maximum (of log2 units) and sum
    uint64_t q_batch, q_head, table_stride, n_pages;
    uint32_t batch, q_heads, kv_heads, group, tiles, splits, page_shift, positions;  // positions: table_width * page_size
    uint32_t class_shift;  // kByLength: classes of lengths
    uint32_t slots;        // kEvenly: chunks that there is room for
    uint32_t *cuts;        // kEvenly: [batch][2]: a sequence's first chunk, and how many it has
    float scale;  // times log2 e
};

struct Range {
    uint32_t start, len, base;  // base: start down to a multiple of the step
    uint32_t steps;
};

__device__ __forceinline__ Range range_of(const AttnParams &p, int32_t len, int32_t start) {
    Range r;
    r.len = min(static_cast<uint32_t>(max(len, 0)), p.positions);
    r.start = min(static_cast<uint32_t>(max(start, 0)), r.len);
    r.base = r.start & ~(kStep - 1);
    r.steps = r.len > r.start ? (r.len - r.base + kStep - 1) / kStep : 0;
    return r;
}

// The lengths of up to 64 kSets sequences in a wave's lanes.
template <int kSets>
struct Lanes {
    int32_t len[kSets], start[kSets];
    uint32_t span[kSets];
    bool have[kSets];

    __device__ __forceinline__ Lanes(const AttnParams &p, uint32_t lane) {
#pragma unroll
        for (int g = 0; g < kSets; ++g) {
            const uint32_t i = 64 * g + lane, at = min(i, p.batch - 1);
            len[g] = p.lens[at];
            start[g] = p.starts ? p.starts[at] : 0;
            have[g] = i < p.batch;
        }
#pragma unroll
        for (int g = 0; g < kSets; ++g) {
            const uint32_t l = min(static_cast<uint32_t>(max(len[g], 0)), p.positions);
            const uint32_t s = min(static_cast<uint32_t>(max(start[g], 0)), l);
            span[g] = have[g] && l > s ? l - (s & ~(kStep - 1)) : 0;
        }
    }
};

struct Sequence {
    uint32_t b;
    int32_t len, start;
};

// The sequence of this rank by length, longest first, found by every wave for
// itself: a ballot for each bit of the lengths' classes keeps the half in which
// the rank lies.  Sequences of a class go in their order.
template <int kSets>
__device__ __forceinline__ Sequence sequence_of(const AttnParams &p, uint32_t rank, uint32_t lane) {
    const Lanes<kSets> lanes(p, lane);
    uint64_t left[kSets];
#pragma unroll
    for (int g = 0; g < kSets; ++g) left[g] = __ballot(lanes.have[g]);
#pragma unroll
    for (int bit = kClassBits - 1; bit >= 0; --bit) {
        uint64_t set[kSets];
        uint32_t n = 0;
#pragma unroll
        for (int g = 0; g < kSets; ++g) {
            const uint32_t key = min(lanes.span[g] >> p.class_shift, (1u << kClassBits) - 1);
            set[g] = left[g] & __ballot(key >> bit & 1u);
            n += __popcll(set[g]);
        }
        const bool in = rank < n;
        rank -= in ? 0 : n;
#pragma unroll
        for (int g = 0; g < kSets; ++g) left[g] = in ? set[g] : left[g] & ~set[g];
    }
    Sequence found = {0, 0, 0};
#pragma unroll
    for (int g = 0; g < kSets; ++g) {
        const uint32_t n = __popcll(left[g]);
        const uint32_t before = __builtin_amdgcn_mbcnt_hi(left[g] >> 32, __builtin_amdgcn_mbcnt_lo(left[g], 0));
        const uint64_t mine = __ballot((left[g] >> lane & 1u) && before == rank);
        if (mine) {  // of one set at most: past it the rank wraps below zero
            const uint32_t at = __builtin_ctzll(mine);
            found = {64 * g + at, __builtin_amdgcn_readlane(lanes.len[g], at), __builtin_amdgcn_readlane(lanes.start[g], at)};
        }
        rank -= n;
    }
    return found;
}

// Lane i receives op over lanes 0..i (op(0, x) = x): shifts inside rows of 16
// lanes, then each row's last value to the rows above.
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), kCtrl, kRows, 0xF, false));
}

template <class Op>
__device__ __forceinline__ uint32_t wave_scan(uint32_t x, Op op) {
    x = op(x, dpp<0x111, 0xF>(x));
    x = op(x, dpp<0x112, 0xF>(x));
    x = op(x, dpp<0x114, 0xF>(x));
    x = op(x, dpp<0x118, 0xF>(x));
    x = op(x, dpp<0x142, 0xA>(x));
    return op(x, dpp<0x143, 0xC>(x));
}

struct Cut {
    Sequence seq;
    uint32_t chunk, chunks;  // chunks: 0 past the last sequence's
};

// The chunk in this slot where all sequences are cut to one length: as many
// units as let p.slots - p.batch chunks hold them all, or p.splits for each
// sequence where the longest is within an eighth of the mean.  A sequence's last
// chunk need not be full, and an empty sequence has an empty one: hence p.batch
// more.
template <int kSets>
__device__ __forceinline__ Cut cut_of(const AttnParams &p, uint32_t slot, uint32_t lane) {
    const Lanes<kSets> lanes(p, lane);
    uint32_t units[kSets], sum = 0, most = 0;
#pragma unroll
    for (int g = 0; g < kSets; ++g) {
        units[g] = (lanes.span[g] + kMinChunk - 1) / kMinChunk;
        sum += units[g];
        most = max(most, units[g]);
    }
    const auto add = [](uint32_t a, uint32_t b) { return a + b; };
    const auto larger = [](uint32_t a, uint32_t b) { return max(a, b); };
    sum = __builtin_amdgcn_readlane(wave_scan(sum, add), 63);
    most = __builtin_amdgcn_readlane(wave_scan(most, larger), 63);
    const uint32_t full = most * p.batch - sum <= sum / 8 ? p.batch * p.splits : p.slots - p.batch, each = max((sum + full - 1) / full, 1u);
    Cut found = {};
    uint32_t first = 0;
#pragma unroll
    for (int g = 0; g < kSets; ++g) {
        const uint32_t n = lanes.have[g] ? max((units[g] + each - 1) / each, 1u) : 0;
        const uint32_t end = first + wave_scan(n, add);
        const uint64_t mine = __ballot(slot < end && slot >= end - n);
        if (mine) {
            const uint32_t at = __builtin_ctzll(mine);
            found.seq = {64 * g + at, __builtin_amdgcn_readlane(lanes.len[g], at), __builtin_amdgcn_readlane(lanes.start[g], at)};
            found.chunks = __builtin_amdgcn_readlane(n, at);
            found.chunk = slot - (__builtin_amdgcn_readlane(end, at) - found.chunks);
        }
        first = __builtin_amdgcn_readlane(end, 63);
    }
    return found;
}

// Waves of a SIMD that the registers are held to (without it the compiler takes
// more and leaves one or two): 8 x 32,768 positions in E4M3 101 -> 99 us, 32 x
// 2,048 BF16 positions of 8 heads of 64 29.2 -> 28.1 us; BF16 heads of 256 are
// left one wave, as two spill: 8 x 8,192 of 8 heads 94 us against 118.
constexpr int waves_for(int dim, bool e4m3) { return dim == 64 ? 4 : dim == 128 ? (e4m3 ? 4 : 3) : e4m3 ? 2 : 1; }

template <int kDim, bool kE4M3, Order kOrder>
__global__ void __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(waves_for(kDim, kE4M3))))
attend_kernel(AttnParams p) {
    constexpr int kPiece = kDim / 16;              // values of a V row in a lane; tiles of out^T
    constexpr int kKChunks = kDim / 32;            // matrix instructions over d
    constexpr int kKLoads = kE4M3 ? kDim / 64 : kKChunks;  // 16-byte loads of a K row in a lane
    constexpr int kVWords = kPiece * (kE4M3 ? 1 : 2) / 4;  // dwords of a V piece
    __shared__ int32_t s_page[kMaxChunk / kMinPage + 1];
    __shared__ float s_stat[kWaves][2][kHeadTile];
    extern __shared__ __attribute__((aligned(16))) float s_out[];  // [kWaves][heads of a tile][kDim + kPad]

    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // chunks of all heads of all sequences before the next chunks: workgroups
    // go round the 8 XCDs, and the first chunks, which every sequence has,
    // spread over all of them
    const uint32_t units = p.batch * p.kv_heads * p.tiles;
    const uint32_t split = kOrder == kAsGiven ? blockIdx.x / units : 0;
    uint32_t rest = blockIdx.x - split * units;
    // workgroups i and i + 256 share a compute unit: every other 256 go from the
    // shorter of their sequences to the longer
    if (kOrder == kByLength && rest / kComputeUnits % 2 == 0) {
        const uint32_t turn = rest / kComputeUnits * kComputeUnits;
        rest = turn + min(turn + kComputeUnits, units) - 1 - rest;
    }
    const uint32_t tile = rest % p.tiles;
    rest /= p.tiles;
    const uint32_t h = rest % p.kv_heads;
    rest /= p.kv_heads;
    const uint32_t heads = min(kHeadTile, p.group - tile * kHeadTile);
    const uint32_t head0 = h * p.group + tile * kHeadTile;
    const uint32_t out_heads = min(kHeadTile, p.group);  // as the host sizes s_out
    const bool single = kOrder == kByLength || (kOrder == kAsGiven && p.splits == 1);
    Sequence seq = {rest, 0, 0};
    Cut cut = {};
    if (kOrder == kAsGiven) {
        seq.len = p.lens[rest];
        seq.start = p.starts ? p.starts[rest] : 0;
    } else if (kOrder == kByLength) {
        seq = p.batch <= 64 ? sequence_of<1>(p, rest, lane) : sequence_of<kLaneSequences / 64>(p, rest, lane);
    } else {
        cut = p.batch <= 64 ? cut_of<1>(p, rest, lane) : cut_of<kLaneSequences / 64>(p, rest, lane);
        if (cut.chunks == 0) return;
        seq = cut.seq;
        if (cut.chunk == 0 && h == 0 && tile == 0 && threadIdx.x == 0) {
            p.cuts[2 * seq.b] = rest;
            p.cuts[2 * seq.b + 1] = cut.chunks;
        }
    }
    const uint32_t b = seq.b;
    const Range range = range_of(p, seq.len, seq.start);
    if (kOrder == kAsGiven)
        cut = {seq, split, min(p.splits, (range.steps + kMinChunk / kStep - 1) / (kMinChunk / kStep))};
    else if (kOrder == kByLength)
        cut = {seq, 0, 1};
    if (kOrder == kAsGiven && !single && cut.chunk >= cut.chunks) {  // nothing here: the join gives it no weight
        for (uint32_t g = threadIdx.x; g < heads; g += 64 * kWaves) {
            float *to = p.stats + 2 * ((uint64_t{b} * p.q_heads + head0 + g) * p.splits + split);
            to[0] = -INFINITY;
            to[1] = 0;
        }
        return;
    }
    // the sequence's steps over its chunks, the first ones with one more; a single chunk may be empty
    const uint32_t chunks = max(cut.chunks, 1u), each = range.steps / chunks, more = range.steps - each * chunks;
    const uint32_t c0 = range.base + (cut.chunk * each + min(cut.chunk, more)) * kStep;
    const uint32_t c1 = max(c0, min(c0 + (each + (cut.chunk < more)) * kStep, range.len));

    // the chunk's pages; -1 masks
    const uint32_t first = c0 >> p.page_shift;
    const uint32_t n_pages = c1 > c0 ? ((c1 - 1) >> p.page_shift) - first + 1 : 0;
    const int32_t *table = p.table + b * p.table_stride + first;
    for (uint32_t i = threadIdx.x; i < n_pages; i += 64 * kWaves) {
        const int32_t e = table[i];
        s_page[i] = e >= 0 && static_cast<uint64_t>(e) < p.n_pages ? e : -1;
    }

    // Q^T: head r, d in the order in which K's loads give them
    const bool have = r < heads;
    const uint16_t *qp = p.q + b * p.q_batch + (head0 + (have ? r : 0)) * p.q_head;
    bf8 qf[kKChunks];
#pragma unroll
    for (int i = 0; i < kKChunks; ++i) {
        const uint32_t d = kE4M3 ? 64 * (i / 2) + 16 * q + 8 * (i & 1) : 32 * i + 8 * q;
        qf[i] = __builtin_bit_cast(bf8, have ? load8(qp + d) : v4u{0, 0, 0, 0});
    }
    const float scale = kE4M3 ? p.scale * p.k.scale[h] : p.scale;
    const uint8_t *kb = p.k.base + h * p.k.head, *vb = p.v.base + h * p.v.head;
    const uint32_t in_page = (1u << p.page_shift) - 1;
    __syncthreads();

    // K rows of a step: lane r has position r of each half
    v4u kr[2][kKLoads];
    auto load_k = [&](uint32_t p0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t pos = min(p0 + 16 * t + r, c1 - 1);
            const int32_t page = max(s_page[(pos >> p.page_shift) - first], 0);
            const uint8_t *row = kb + static_cast<uint64_t>(page) * p.k.page + uint64_t{pos & in_page} * p.k.row + 16 * q;
#pragma unroll
            for (int i = 0; i < kKLoads; ++i) kr[t][i] = *reinterpret_cast<const v4u *>(row + 64 * i);
        }
    };
    // V rows of a step: positions 4 q + 0..3 of each half (of one page: pages
    // hold multiples of 8); live: those that count
    typedef uint32_t VRow __attribute__((ext_vector_type(kVWords)));
    typedef VRow VRowInMemory __attribute__((aligned(4)));
    VRow vr[8];
    bool live[8];
    auto load_v = [&](uint32_t p0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t pos0 = p0 + 16 * t + 4 * q, at0 = min(pos0, c1 - 1);
            const int32_t page = s_page[(at0 >> p.page_shift) - first];
            const uint8_t *rows = vb + static_cast<uint64_t>(max(page, 0)) * p.v.page + r * (kVWords * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t pos = pos0 + i, at = min(pos, c1 - 1);
                live[4 * t + i] = pos >= range.start && pos < c1 && page >= 0;
                const uint8_t *row = rows + uint64_t{at & in_page} * p.v.row;
                vr[4 * t + i] = *reinterpret_cast<const VRowInMemory *>(row);
            }
        }
    };

    float m = -INFINITY, l = 0;  // m over all lanes of a head, l over this lane's positions
    f4 acc[kPiece] = {};
    uint32_t p0 = c0 + wave * kStep;
    if (p0 < c1) {
        load_k(p0);
        // K's loads before V's, as in the loop: a wave waits for the oldest ones, and
        // otherwise for V's at the head of every step.  The two empty statements, which
        // differ, keep the compiler from joining both loads of V at that head.
        __builtin_amdgcn_sched_barrier(0);
        load_v(p0);
        asm volatile("; V of the first step" ::: "memory");
    }
    // The registers of K and V are loaded again as soon as they are used up.  The
    // last step, which loads nothing, is a copy of its own: where the loads are left
    // out on a condition, the wait for V has to be one for the next K too (one
    // sequence of 65,536 positions in E4M3 30.9 us, so 26.7; 32 x 2,048 of 8 BF16
    // heads of 64 23.4, so 21.4; where the last step loads in vain 27.4 and 21.9).
    auto step = [&](uint32_t next, auto more) {
        constexpr bool kMore = decltype(more)::value;
        f4 s[2] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < kKChunks; ++i) {
                v4u kw;
                if (kE4M3)
                    kw = i & 1 ? from_e4m3x8(kr[t][i / 2].z, kr[t][i / 2].w) : from_e4m3x8(kr[t][i / 2].x, kr[t][i / 2].y);
                else
                    kw = kr[t][kE4M3 ? 0 : i];
                s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, kw), qf[i], s[t], 0, 0, 0);
            }
        if (kMore) load_k(next);
        float x[8], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = live[i] ? s[i / 4][i & 3] * scale : -INFINITY;
            top = fmaxf(top, x[i]);
        }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m_new = fmaxf(m, top);
        const float ref = m_new == -INFINITY ? 0.0f : m_new;  // nothing but masked positions so far
        const float fade = exp2_(m - ref);
        m = m_new;
        float w[8];
        l *= fade;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = exp2_(x[i] - ref);
            l += w[i];
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[i] = kE4M3 ? pack2(w[2 * i], w[2 * i + 1]) : cut2(w[2 * i], w[2 * i + 1]);
            lo[i] = pack2(w[2 * i] - __builtin_bit_cast(float, hi[i] << 16),
                          w[2 * i + 1] - __builtin_bit_cast(float, hi[i] & 0xFFFF0000u));
            if (!kE4M3) lo[i] = at_least2(lo[i], kLeastPart);
        }
        const bf8 w_hi = __builtin_bit_cast(bf8, v4u{hi[0], hi[1], hi[2], hi[3]});
        const bf8 w_lo = __builtin_bit_cast(bf8, v4u{lo[0], lo[1], lo[2], lo[3]});
        // a masked row may hold anything, and 0 times NaN is NaN
        const bool all = live[0] && live[1] && live[2] && live[3] && live[4] && live[5] && live[6] && live[7];
        if (!__all(all)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) vr[i] = live[i] ? vr[i] : VRow(0);
        }
#pragma unroll
        for (int j = 0; j < kPiece; j += 2) {
            // values j and j + 1 of the eight rows
            uint32_t pair[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (kE4M3)
                    pair[i] = j & 2 ? from_e4m3<true>(vr[i][j / 4]) : from_e4m3<false>(vr[i][j / 4]);
                else
                    pair[i] = vr[i][kE4M3 ? 0 : j / 2];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t sel = e ? 0x07060302u : 0x05040100u;
                const bf8 a = __builtin_bit_cast(
                    bf8, v4u{__builtin_amdgcn_perm(pair[1], pair[0], sel), __builtin_amdgcn_perm(pair[3], pair[2], sel),
                             __builtin_amdgcn_perm(pair[5], pair[4], sel), __builtin_amdgcn_perm(pair[7], pair[6], sel)});
                f4 o = acc[j + e];
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] *= fade;
                o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, w_hi, o, 0, 0, 0);
                acc[j + e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, w_lo, o, 0, 0, 0);
            }
        }
        if (kMore) {
            load_v(next);
            asm volatile("; V of the next step" ::: "memory");
        }
    };
    if (p0 < c1) {
        for (uint32_t next = p0 + kWaves * kStep; next < c1; next += kWaves * kStep) step(next, std::true_type());
        step(0, std::false_type());
    }

    // join the waves
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (q == 0) {
        s_stat[wave][0][r] = m;
        s_stat[wave][1][r] = l;
    }
    // acc[j][c]: d = (4 q + c) * kPiece + j
    if (have) {
        float *to = s_out + (wave * out_heads + r) * (kDim + kPad) + 4 * q * kPiece;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < kPiece; j += 4)
                *reinterpret_cast<f4 *>(to + c * kPiece + j) = f4{acc[j][c], acc[j + 1][c], acc[j + 2][c], acc[j + 3][c]};
    }
    __syncthreads();
    const float v_scale = kE4M3 ? p.v.scale[h] : 1.0f;
    for (uint32_t i = threadIdx.x; i < heads * kDim; i += 64 * kWaves) {
        const uint32_t g = i / kDim, d = i % kDim;
        float top = -INFINITY;
#pragma unroll
        for (uint32_t k = 0; k < kWaves; ++k) top = fmaxf(top, s_stat[k][0][g]);
        const float ref = top == -INFINITY ? 0.0f : top;
        float sum = 0, o = 0;
#pragma unroll
        for (uint32_t k = 0; k < kWaves; ++k) {
            const float f = exp2_(s_stat[k][0][g] - ref);
            sum += s_stat[k][1][g] * f;
            o += s_out[(k * out_heads + g) * (kDim + kPad) + d] * f;
        }
        o *= v_scale;
        const uint64_t row = uint64_t{b} * p.q_heads + head0 + g;
        if (single) {
            p.out[row * kDim + d] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(sum == 0 ? 0.0f : o / sum));
            if (d == 0 && p.lse) p.lse[row] = (top + __builtin_amdgcn_logf(sum)) * kLn2;
        } else {
            const uint64_t at = kOrder == kEvenly ? uint64_t{head0 + g} * p.slots + rest : row * p.splits + split;
            p.part[at * kDim + d] = o;
            if (d == 0) {
                p.stats[2 * at] = top;
                p.stats[2 * at + 1] = sum;
            }
        }
    }
}

// One workgroup joins the chunks of one query head: every wave's lanes read the
// chunks' maxima and sums side by side, kDim / 4 lanes take four values each of
// every kGroups-th chunk, and LDS adds what they have.  Bound by latency: the
// maxima, the sums and the first chunks' values are loaded without waiting for
// one another (a chunk without positions has left its values unwritten; they
// are read and given no weight).
constexpr uint32_t kJoinThreads = 256;

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int i = 32; i; i >>= 1) v = fmaxf(v, __shfl_xor(v, i));
    return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int i = 32; i; i >>= 1) v += __shfl_xor(v, i);
    return v;
}

template <int kDim>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttnParams p) {
    constexpr uint32_t kQuads = kDim / 4, kGroups = kJoinThreads / kQuads;
    __shared__ f4 s_part[kGroups][kQuads];
    const uint64_t row = blockIdx.x;
    const uint32_t lane = threadIdx.x & 63u, d = threadIdx.x % kQuads, group = threadIdx.x / kQuads;
    uint64_t at = row * p.splits;
    uint32_t splits = p.splits;
    if (p.cuts) {
        const uint32_t b = static_cast<uint32_t>(row / p.q_heads);
        // within the workspace also where the lengths were written to during the call
        const uint32_t first = min(p.cuts[2 * b], p.slots);
        at = (row - uint64_t{b} * p.q_heads) * p.slots + first;
        splits = min(p.cuts[2 * b + 1], p.slots - first);
    }
    const v2f *stats = reinterpret_cast<const v2f *>(p.stats) + at;
    const f4 *part = reinterpret_cast<const f4 *>(p.part + at * kDim) + d;
    constexpr int kAhead = 4;
    v2f first = {-INFINITY, 0};
    if (lane < splits) first = stats[lane];
    f4 v[kAhead] = {};
    float m[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
        const uint32_t i = group + a * kGroups;
        m[a] = -INFINITY;
        if (i < splits) {
            m[a] = stats[i].x;
            v[a] = part[uint64_t{i} * kQuads];
        }
    }
    float top = first.x;
    for (uint32_t i = lane + 64; i < splits; i += 64) top = fmaxf(top, stats[i].x);
    top = wave_max(top);
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = first.y * exp2_(first.x - ref);
    for (uint32_t i = lane + 64; i < splits; i += 64) sum += stats[i].y * exp2_(stats[i].x - ref);
    sum = wave_sum(sum);
    f4 o = {};
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
        const float f = exp2_(m[a] - ref);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += m[a] == -INFINITY ? 0.0f : v[a][j] * f;
    }
    for (uint32_t i = group + kAhead * kGroups; i < splits; i += kGroups) {
        const float mi = stats[i].x, f = exp2_(mi - ref);
        const f4 w = part[uint64_t{i} * kQuads];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += mi == -INFINITY ? 0.0f : w[j] * f;
    }
    s_part[group][d] = o;
    __syncthreads();
    if (threadIdx.x < kQuads) {
#pragma unroll
        for (uint32_t g = 1; g < kGroups; ++g) {
            const f4 v = s_part[g][d];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] += v[j];
        }
        const float inv = sum == 0 ? 0.0f : 1.0f / sum;
        v2u out;
        out.x = pack2(o[0] * inv, o[1] * inv);
        out.y = pack2(o[2] * inv, o[3] * inv);
        *reinterpret_cast<v2u *>(p.out + row * kDim + 4 * d) = out;
        if (threadIdx.x == 0 && p.lse) p.lse[row] = (top + __builtin_amdgcn_logf(sum)) * kLn2;
    }
}

// ---- Host ------------------------------------------------------------------

df11_status append(const df11_paged_cache *c, const uint16_t *k, uint64_t k_token, uint64_t k_head, const uint16_t *v,
                   uint64_t v_token, uint64_t v_head, const int64_t *slots, uint64_t tokens, void *hip_stream) {
    const df11_status rc = check_cache(c);
    if (rc != DF11_OK) return rc;
    if (tokens == 0) return DF11_OK;
    if (!k || !v || !slots || tokens > 0x7FFFFFFFu || (reinterpret_cast<uintptr_t>(slots) & 7u) ||
        ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 1u))
        return DF11_E_INVALID_ARG;
    for (uint64_t s : {k_token, k_head, v_token, v_head})
        if (s > kMaxStride) return DF11_E_INVALID_ARG;
    if (span(tokens, k_token) + span(c->kv_heads, k_head) >= kMaxExtent ||
        span(tokens, v_token) + span(c->kv_heads, v_head) >= kMaxExtent)
        return DF11_E_INVALID_ARG;
    AppendParams p;
    p.k = k_of(c);
    p.v = v_of(c);
    p.ks = k;
    p.vs = v;
    p.k_token = k_token;
    p.k_head = k_head;
    p.v_token = v_token;
    p.v_head = v_head;
    p.slots = slots;
    p.per_token = c->kv_heads * (c->head_dim / 8);
    p.dim_shift = log2_of(c->head_dim / 8);
    p.page_shift = log2_of(c->page_size);
    p.n_slots = c->n_pages * c->page_size;
    p.lanes = tokens * p.per_token;
    auto fn = c->dtype == DF11_CACHE_E4M3 ? append_kernel<true> : append_kernel<false>;
    const uint32_t grid = static_cast<uint32_t>(std::min<uint64_t>((p.lanes + 255) / 256, 1u << 20));
    return launched(launch(fn, grid, 256, 0, static_cast<hipStream_t>(hip_stream), p));
}

// Chunks of a sequence.  The device cuts what a sequence really holds, so the
// page table's width only bounds them: as many as give each of 256 compute
// units a workgroup, no more than chunks of kMinChunk, and enough that none
// exceeds kMaxChunk; none where the table holds at most 256 positions (a second
// kernel takes longer than the second step of a wave).  Measured with 256, 512 and
// 1,024 workgroups wanted: 8 x 32,768 BF16 positions of 8 heads (1.07 GB) 188, 188
// and 190 us; one sequence of 65,536 52.1, 53.2 and 55.9; 16 windows of 1,024 over
// 4 heads of 256 17.3, 20.2 and 22.7.
constexpr uint64_t kWantGroups = kComputeUnits;

uint32_t splits_of(uint64_t batch, uint32_t kv_heads, uint32_t tiles, uint64_t positions) {
    if (positions <= 2 * kMinChunk) return 1;
    const uint64_t units = std::max<uint64_t>(batch * kv_heads * tiles, 1);
    const uint64_t want = (kWantGroups + units - 1) / units;
    const uint64_t most = (positions + kMinChunk - 1) / kMinChunk, least = (positions + kMaxChunk - 1) / kMaxChunk;
    return static_cast<uint32_t>(std::max(std::min(want, most), std::max<uint64_t>(least, 1)));
}

// Chunks that there is room for where all sequences are cut to one length; 0: each
// is cut by itself.  Cut by itself, a short sequence's chunks end early and leave
// their compute units idle; cut evenly, a longer start (all lengths have to be
// read and summed) and a longer join.  So only where the chunks would be long.
// Measured by itself and evenly, BF16 sequences of 8 heads of 128: 8 ragged ones up
// to 32,768 119 and 92 us, up to 8,192 34.4 and 28.3, 8 of the same 32,768 185.4 and
// 185.5, of the same 8,192 52.2 and 52.5; with chunks of 1,024, 4 ragged ones up to
// 8,192, 16.5 and 17.2.  Ragged sequences get up to four chunks for each compute
// unit, none under kMinEvenChunk (8 ragged up to 32,768: 104 us with one, 94 with
// four, 97 with eight); nearly equal ones as many as kAsGiven (8 of the same 32,768
// 190 us with four).
constexpr uint64_t kMinEven = 2048, kMinEvenChunk = 1024, kWantEven = 4 * kComputeUnits;

uint64_t slots_of(uint64_t batch, uint32_t kv_heads, uint32_t tiles, uint64_t positions, uint32_t splits) {
    if (splits <= 1 || batch < 2 || batch > kLaneSequences || positions / splits < kMinEven || positions >= (1u << 30)) return 0;
    const uint64_t units = batch * kv_heads * tiles;
    return batch * (std::max<uint64_t>(splits, std::min((kWantEven + units - 1) / units, positions / kMinEvenChunk)) + 1);
}

// By length where compute units share whole sequences: 64 ragged ones of 8 BF16 heads
// of 128 up to 1,024 positions 33.8 us as given, 28.4 by length, up to 2,048 59 and 51,
// 48 up to 1,024 26.1 and 21.2; 64 of the same 512 23.6 and 24.0.  Ranking takes the
// longer the more sequences there are and gains nothing where all are short: 64 ragged
// ones up to 256 11.6 and 11.6, 256 up to 256 27.8 and 30.6, up to 1,024 107 and 99.
Order order_of(uint64_t batch, uint64_t units, uint64_t positions, uint32_t splits, uint64_t slots) {
    if (slots) return kEvenly;
    return splits == 1 && units > kComputeUnits && batch <= kLaneSequences && positions >= std::max<uint64_t>(512, 4 * batch)
               ? kByLength
               : kAsGiven;
}

uint64_t attention_workspace(uint64_t batch, uint64_t q_heads, uint32_t head_dim, uint32_t splits, uint64_t slots) {
    if (splits <= 1) return 0;
    return (slots ? slots : batch * splits) * q_heads * (head_dim + 2) * sizeof(float) + (slots ? 2 * batch * sizeof(uint32_t) : 0);
}

uint64_t workgroups(uint64_t batch, uint32_t kv_heads, uint32_t tiles, uint32_t splits, uint64_t slots) {
    return (slots ? slots : batch * splits) * kv_heads * tiles;
}

// Whether both kernels' work items fit a launch, which holds fewer than 2^32
// (the counts that can get here stay within 64 bits).
bool launchable(uint64_t batch, uint64_t q_heads, uint32_t kv_heads, uint32_t tiles, uint32_t splits, uint64_t slots) {
    constexpr uint64_t kItems = uint64_t{1} << 32;
    return workgroups(batch, kv_heads, tiles, splits, slots) < kItems / (64 * kWaves) &&
           (splits == 1 || batch * q_heads < kItems / kJoinThreads);
}

bool attention_sizes_ok(uint64_t batch, uint64_t q_heads, uint32_t kv_heads, uint32_t page_size, uint64_t width) {
    return batch <= (1u << 24) && kv_heads > 0 && q_heads > 0 && q_heads <= (1u << 20) && q_heads % kv_heads == 0 &&
           width > 0 && width <= 0x7FFFFFFFu / page_size;
}

template <int kDim>
auto attend_of(bool e4m3, Order order) {
    switch (order) {
        case kByLength: return e4m3 ? attend_kernel<kDim, true, kByLength> : attend_kernel<kDim, false, kByLength>;
        case kEvenly: return e4m3 ? attend_kernel<kDim, true, kEvenly> : attend_kernel<kDim, false, kEvenly>;
        default: return e4m3 ? attend_kernel<kDim, true, kAsGiven> : attend_kernel<kDim, false, kAsGiven>;
    }
}

df11_status attention(const df11_paged_cache *c, const uint16_t *q, uint64_t batch, uint64_t q_heads, uint64_t q_batch,
                      uint64_t q_head, const int32_t *table, uint64_t table_stride, uint64_t width, const int32_t *lens,
                      const int32_t *starts, float scale, uint16_t *out, float *lse, void *workspace,
                      uint64_t workspace_bytes, void *hip_stream) {
    const df11_status rc = check_cache(c);
    if (rc != DF11_OK) return rc;
    if (!attention_sizes_ok(batch, q_heads, c->kv_heads, c->page_size, width) || table_stride < width ||
        table_stride > kMaxStride || q_batch > kMaxStride || q_head > kMaxStride ||
        span(batch, table_stride) >= kMaxExtent || span(batch, q_batch) + span(q_heads, q_head) >= kMaxExtent)
        return DF11_E_INVALID_ARG;
    if (batch == 0) return DF11_OK;
    if (!q || !table || !lens || !out || (reinterpret_cast<uintptr_t>(q) & 1u) || !aligned16(out) ||
        ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(starts) |
          reinterpret_cast<uintptr_t>(lse)) & 3u) ||
        !aligned16(workspace))
        return DF11_E_INVALID_ARG;
    AttnParams p;
    p.k = k_of(c);
    p.v = v_of(c);
    p.q = q;
    p.table = table;
    p.lens = lens;
    p.starts = starts;
    p.out = out;
    p.lse = lse;
    p.q_batch = q_batch;
    p.q_head = q_head;
    p.table_stride = table_stride;
    p.n_pages = c->n_pages;
    p.batch = static_cast<uint32_t>(batch);
    p.q_heads = static_cast<uint32_t>(q_heads);
    p.kv_heads = c->kv_heads;
    p.group = p.q_heads / p.kv_heads;
    p.tiles = (p.group + kHeadTile - 1) / kHeadTile;
    p.page_shift = log2_of(c->page_size);
    p.positions = static_cast<uint32_t>(width * c->page_size);
    p.scale = scale * kLog2e;
    p.splits = splits_of(batch, p.kv_heads, p.tiles, p.positions);
    const uint64_t units = batch * p.kv_heads * p.tiles, rows = batch * q_heads;
    p.slots = static_cast<uint32_t>(slots_of(batch, p.kv_heads, p.tiles, p.positions, p.splits));
    const bool even = p.slots != 0;
    p.class_shift = p.positions >> kClassBits ? log2_of(p.positions - 1) + 1 - kClassBits : 0;
    if (!launchable(batch, q_heads, p.kv_heads, p.tiles, p.splits, p.slots)) return DF11_E_INVALID_ARG;
    if (workspace_bytes < attention_workspace(batch, q_heads, c->head_dim, p.splits, p.slots)) return DF11_E_BUFFER_TOO_SMALL;
    if (p.splits > 1 && !workspace) return DF11_E_INVALID_ARG;
    p.part = static_cast<float *>(workspace);
    const uint64_t chunks = even ? p.slots : p.splits > 1 ? batch * p.splits : 0;
    p.stats = p.part + chunks * q_heads * c->head_dim;
    p.cuts = even ? reinterpret_cast<uint32_t *>(p.stats + chunks * q_heads * 2) : nullptr;
    const uint64_t groups = workgroups(batch, p.kv_heads, p.tiles, p.splits, p.slots);
    const bool e4m3 = c->dtype == DF11_CACHE_E4M3;
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    const Order order = order_of(batch, units, p.positions, p.splits, p.slots);
    auto fn = c->head_dim == 64    ? attend_of<64>(e4m3, order)
              : c->head_dim == 128 ? attend_of<128>(e4m3, order)
                                   : attend_of<256>(e4m3, order);
    hipError_t err = launch(fn, static_cast<uint32_t>(groups), 64 * kWaves,
                            kWaves * std::min(kHeadTile, p.group) * (c->head_dim + kPad) * sizeof(float), st, p);
    if (err == hipSuccess && p.splits > 1)
        err = launch(c->head_dim == 64    ? join_kernel<64>
                     : c->head_dim == 128 ? join_kernel<128>
                                          : join_kernel<256>,
                     static_cast<uint32_t>(rows), kJoinThreads, 0, st, p);
    return launched(err);
}

}  // namespace

extern "C" df11_status df11_paged_append(const df11_paged_cache *cache, const uint16_t *k, uint64_t k_token_stride,
                                         uint64_t k_head_stride, const uint16_t *v, uint64_t v_token_stride,
                                         uint64_t v_head_stride, const int64_t *slots, uint64_t tokens,
                                         void *hip_stream) {
    return df11i::guarded([&] {
        return append(cache, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, slots, tokens, hip_stream);
    });
}

extern "C" uint64_t df11_paged_attention_workspace_bytes(uint64_t batch, uint64_t q_heads, uint32_t kv_heads,
                                                         uint32_t head_dim, uint32_t page_size, uint64_t table_width) {
    if (!page_ok(page_size) || !attention_sizes_ok(batch, q_heads, kv_heads, page_size, table_width)) return 0;
    const uint32_t group = static_cast<uint32_t>(q_heads / kv_heads);
    const uint32_t tiles = (group + kHeadTile - 1) / kHeadTile;
    const uint64_t positions = table_width * page_size;
    const uint32_t splits = splits_of(batch, kv_heads, tiles, positions);
    const uint64_t slots = slots_of(batch, kv_heads, tiles, positions, splits);
    if (!launchable(batch, q_heads, kv_heads, tiles, splits, slots)) return 0;
    return attention_workspace(batch, q_heads, head_dim, splits, slots);
}

extern "C" df11_status df11_paged_attention(const df11_paged_cache *cache, const uint16_t *q, uint64_t batch,
                                            uint64_t q_heads, uint64_t q_batch_stride, uint64_t q_head_stride,
                                            const int32_t *page_table, uint64_t table_stride, uint64_t table_width,
                                            const int32_t *lens, const int32_t *starts, float scale, uint16_t *out,
                                            float *lse, void *workspace, uint64_t workspace_bytes, void *hip_stream) {
    return df11i::guarded([&] {
        return attention(cache, q, batch, q_heads, q_batch_stride, q_head_stride, page_table, table_stride, table_width,
                         lens, starts, scale, out, lse, workspace, workspace_bytes, hip_stream);
    });
}
