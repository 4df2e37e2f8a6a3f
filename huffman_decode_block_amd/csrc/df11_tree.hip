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

// Scores s = scale q . k of a row over the positions that it reads, out = sum exp(s) v /
// sum exp(s), in one pass: a row keeps a reference near its largest score so far, the
// sum of exp(s - reference) and of the weighted values, all in 32 bits.  S^T = K Q^T and
// out^T = V^T P^T by matrix instructions: a lane then has four positions' scores of
// one row, turns them into weights in registers, and those are an operand of the second
// product as they are.  The reference follows only scores that pass it by more than
// kSlack, so that most steps rescale nothing.  No vector register is kept in memory: the
// compiler may store one in front of the instruction that turns the lanes of a finished
// loop on again, and reads back what was there before in those lanes.
constexpr uint32_t kWaves = 4;
constexpr uint32_t kStep = 32;
constexpr uint32_t kMinChunk = kWaves * kStep;
constexpr uint32_t kMaxChunk = 4096;  // positions whose pages LDS holds
constexpr uint32_t kChunkPages = kMaxChunk / kMinPage + 1;
constexpr uint32_t kPad = 4;  // floats between rows in LDS: they start in different banks
constexpr uint32_t kSlots = 2 * kComputeUnits;  // workgroups that run at once
// What looking at masks costs a chunk, in steps: the last chunk gets so many fewer (64
// nodes behind 1,024 positions 22.8 us, with equal chunks 24.8; 4,096 30.1 and 30.6; 8,192
// 33.1 and 32.9).
constexpr uint32_t kMaskedSteps = 3;
constexpr float kSlack = 8;   // powers of two that weights may grow by before their reference follows
// Powers of two by which the reference stays below the largest score of an E4M3 cache: the
// weights become FP16, whose numbers end 2^-25 below 1 and 2^15 above.  A row's largest
// weight is 2^7 to 2^15, and what gets lost is 2^-32 of it, not 2^-25.
constexpr float kLift = 7;

struct TreeParams {
    Pages k, v;
    const uint16_t *q;
    const int32_t *table, *lens, *counts, *starts;
    const int64_t *mask;
    uint16_t *out;
    float *lse;
    float *part;   // [chunks][nodes * q_heads][head_dim]: sums of weighted values
    float *stats;  // [chunks][nodes * q_heads][2]: reference (of log2 units) and sum
    uint32_t *own; // [batch][2]: a sequence's first chunk and how many it has; null: `splits` each
    uint64_t q_batch, q_node, q_head, mask_batch, mask_node, starts_batch, starts_node, table_stride, n_pages;
    uint32_t batch, nodes, q_heads, kv_heads, group, tiles, splits, page_shift, positions;
    uint32_t units;  // kv_heads * chunks
    uint32_t share;  // chunks among which the steps of all sequences are shared, where those have as many as they need
    float scale;     // times log2 e
};

// Bits lo..hi - 1 of 32, both held to [0, 32].
__device__ __forceinline__ uint32_t bits_between(int32_t lo, int32_t hi) {
    const uint32_t l = static_cast<uint32_t>(min(max(lo, 0), 32)), h = static_cast<uint32_t>(min(max(hi, 0), 32));
    const uint64_t below_h = (uint64_t{1} << h) - 1, below_l = (uint64_t{1} << l) - 1;
    return static_cast<uint32_t>(below_h & ~below_l);
}

// Two floats rounded to FP16, and to BF16, by one instruction.
__device__ __forceinline__ uint32_t pack2h(float a, float b) { return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, h2)); }

__device__ __forceinline__ uint32_t pack2b(float a, float b) { return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, bf2)); }

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

// A value's kind as a BF16 number: 1 for infinity, 64 for -infinity, 4096 for NaN,
// 0 for all others; sums of 32 of them tell the kinds apart.
__device__ __forceinline__ uint32_t kind_of(uint32_t bf16) {
    const uint32_t a = bf16 & 0x7FFFu;
    return a < 0x7F80u ? 0u : a > 0x7F80u ? 0x4580u : bf16 & 0x8000u ? 0x4280u : 0x3F80u;
}

template <bool kE4M3>
__device__ __forceinline__ uint32_t kind_at(const uint8_t *row, uint32_t d) {
    if (kE4M3) return (row[d] & 0x7Fu) == 0x7Fu ? 0x4580u : 0u;
    return kind_of(reinterpret_cast<const uint16_t *>(row)[d]);
}

__device__ __forceinline__ float of_counts(float sum) {
    const uint32_t n = static_cast<uint32_t>(sum), plus = n & 63u, minus = n >> 6 & 63u;
    return n >> 12 || (plus && minus) ? NAN : plus ? INFINITY : minus ? -INFINITY : 0.0f;
}

// Four values of a row's output, or of its part in a chunk: `there` where the row has a node.
template <int kDim>
__device__ __forceinline__ void write_out(const TreeParams &p, uint64_t chunk, uint64_t row, uint32_t d, bool there, float top, float total, f4 o) {
    if (!there) {
        top = -INFINITY;
        total = 0;
        o = f4{};
    }
    if (p.splits == 1) {
        if (total == 0) o = f4{};
        const float inv = total == 0 ? 0.0f : 1.0f / total;
        v2u to;
        to.x = pack2b(o[0] * inv, o[1] * inv);
        to.y = pack2b(o[2] * inv, o[3] * inv);
        *reinterpret_cast<v2u *>(p.out + row * kDim + d) = to;
        if (d == 0 && p.lse) p.lse[row] = ((top == -INFINITY ? 0.0f : top) + __builtin_amdgcn_logf(total)) * kLn2;
    } else {
        const uint64_t at = row + chunk * p.nodes * p.q_heads;
        *reinterpret_cast<f4 *>(p.part + at * kDim + d) = o;
        if (d == 0) {
            p.stats[2 * at] = top;
            p.stats[2 * at + 1] = total;
        }
    }
}

// What a workgroup works on: a tile of the rows (row n: node n / group, head n %
// group) of a cache head of a sequence, and a chunk of its positions.
struct Work {
    uint32_t tile, b, h, split;
    uint32_t chunks;  // of the sequence, at most
    int32_t len;      // of the sequence
    uint64_t chunk;   // among those of all sequences, less b: what a row's number lacks to that of its part
    bool none;
};

__device__ __forceinline__ int32_t length_of(const TreeParams &p, uint32_t b) {
    return static_cast<int32_t>(min(static_cast<uint32_t>(max(p.lens[b], 0)), p.positions));
}

// A batch of different lengths: chunks as long as each other, so that a long sequence
// has more of them.  Lane b counts those of sequence b: the steps of all are shared
// among as many chunks as run at once, less half of one for each sequence's last
// (less a quarter: 43.0 us for the first below).  Against as many chunks for each sequence:
// 16 ragged up to 2,048 with 25 nodes 35.9 us in place of 42.2, 8 up to 8,192 47.1 (62.0), 32
// up to 4,096 with 8 nodes 64.2 (75.3); equal lengths pay for the scans and the ends, 16 x
// 2,048 with 25 nodes 49.9 us (49.2), 8 x 32,768 E4M3 with 16 nodes of 64 heads 181 (175).
__device__ __forceinline__ void ragged_work(const TreeParams &p, uint32_t chunk, Work &w) {
    const uint32_t lane = threadIdx.x & 63u, b = min(lane, p.batch - 1);
    const int32_t len = length_of(p, b), start = p.starts ? min(max(p.starts[b * p.starts_batch], 0), len) : 0;
    const uint32_t steps = lane < p.batch ? (static_cast<uint32_t>(len - start) + p.nodes + kStep - 1) / kStep : 0;
    const uint32_t all = __builtin_amdgcn_readlane(df11w::wave_inclusive_scan(steps), 63);
    const uint32_t each = max((all + p.share - 1) / p.share, kMinChunk / kStep);
    const uint32_t mine = (steps + each - 1) / each, to = df11w::wave_inclusive_scan(mine);
    const uint64_t found = __ballot(to - mine <= chunk && chunk < to);
    w.none = found == 0;
    w.b = w.none ? 0 : __builtin_ctzll(found);
    w.chunks = __builtin_amdgcn_readlane(mine, w.b);
    const uint32_t first = __builtin_amdgcn_readlane(to, w.b) - w.chunks;
    w.split = chunk - first;
    w.len = __builtin_amdgcn_readlane(len, w.b);
    w.chunk = uint64_t{chunk} - w.b;
    if (w.split == 0 && w.tile == 0 && w.h == 0 && threadIdx.x == 0) {
        p.own[2 * w.b] = first;
        p.own[2 * w.b + 1] = w.chunks;
    }
}

__device__ __forceinline__ Work work_of(const TreeParams &p) {
    // workgroups go round the 8 XCDs: those of one chunk's tiles, which read the
    // same keys and values, stay on one
    const uint32_t turn = blockIdx.x / (8 * p.tiles), in = blockIdx.x - turn * 8 * p.tiles;
    Work w;
    w.tile = in / 8;
    const uint32_t unit = turn * 8 + (in & 7u);
    w.none = unit >= p.units;
    if (w.none) return w;
    const uint32_t chunk = unit / p.kv_heads;
    w.h = unit - chunk * p.kv_heads;
    if (p.own) {
        ragged_work(p, chunk, w);
    } else {
        w.split = chunk / p.batch;
        w.b = chunk - w.split * p.batch;
        w.chunks = p.splits;
        w.len = length_of(p, w.b);
        w.chunk = uint64_t{w.b} * (p.splits - 1) + w.split;
    }
    // known to be the same in all lanes
    w.tile = __builtin_amdgcn_readfirstlane(w.tile);
    w.h = __builtin_amdgcn_readfirstlane(w.h);
    w.b = __builtin_amdgcn_readfirstlane(w.b);
    w.split = __builtin_amdgcn_readfirstlane(w.split);
    w.chunks = __builtin_amdgcn_readfirstlane(w.chunks);
    w.len = __builtin_amdgcn_readfirstlane(w.len);
    return w;
}

struct Rows {
    uint32_t row0, rows;  // of the tile
    int32_t count, len;   // of the sequence
};

__device__ __forceinline__ Rows rows_of(const TreeParams &p, const Work &w, uint32_t per_tile) {
    Rows r;
    r.row0 = w.tile * per_tile;
    r.rows = min(per_tile, p.nodes * p.group - r.row0);
    r.count = min(max(p.counts ? p.counts[w.b] : INT32_MAX, 0), static_cast<int32_t>(p.nodes));
    r.len = w.len;
    return r;
}

// Where row i of a tile lies among the outputs' rows.
__device__ __forceinline__ uint64_t out_row(const TreeParams &p, const Work &w, const Rows &rows, uint32_t i) {
    const uint32_t n = rows.row0 + i, node = n / p.group;
    return (uint64_t{w.b} * p.nodes + node) * p.q_heads + w.h * p.group + (n - node * p.group);
}

// A lane's row in a tile of 16: its node, the first position that it reads, and whether there is such a node.
struct Row {
    int32_t node, start;
    bool have;
};

__device__ __forceinline__ Row row_of(const TreeParams &p, const Work &w, const Rows &rows, uint32_t i, uint64_t *first) {
    Row r;
    r.node = static_cast<int32_t>(min(rows.row0 + i, p.nodes * p.group - 1) / p.group);
    r.have = i < rows.rows && r.node < rows.count;
    r.start = 0;
    if (p.starts)
        r.start = min(max(p.starts[w.b * p.starts_batch + static_cast<uint32_t>(r.node) * p.starts_node], 0), rows.len);
    // its mask's first word is looked at seldom: LDS keeps it
    if (p.mask) *first = static_cast<uint64_t>(p.mask[w.b * p.mask_batch + static_cast<uint32_t>(r.node) * p.mask_node]);
    return r;
}

// The chunk: positions c0..c1 - 1 of those (from lo on) that any row of the tile
// reads; all rows read those from lo_max to all_hi - 1.
struct Chunk {
    int32_t lo, lo_max, all_hi, c0, c1;
    bool none;
};

__device__ __forceinline__ Chunk chunk_of(const TreeParams &p, const Work &w, const Rows &rows, int32_t lo, int32_t lo_max) {
    const int32_t node_first = static_cast<int32_t>(rows.row0 / p.group), node_last = static_cast<int32_t>((rows.row0 + rows.rows - 1) / p.group);
    const int32_t reach = min(rows.count, p.mask ? rows.count : node_last + 1);
    const int32_t hi = node_first < rows.count ? static_cast<int32_t>(min(static_cast<uint32_t>(rows.len + reach), p.positions)) : 0;
    const int32_t base = lo & ~static_cast<int32_t>(kStep - 1);
    const uint32_t steps = hi > base ? (hi - base + kStep - 1) / kStep : 0;
    const uint32_t chunks = p.own ? w.chunks : min(w.chunks, (steps + kMinChunk / kStep - 1) / (kMinChunk / kStep));
    // the last chunk has steps in which masks are looked at, and gets fewer
    const uint32_t parts = max(chunks, 1u), full = steps + min(kMaskedSteps, steps / parts / 2), each = full / parts, more = full - each * parts;
    Chunk c;
    c.lo = lo;
    c.lo_max = lo_max;
    c.all_hi = p.mask ? rows.len : min(rows.len + min(node_first + 1, rows.count), hi);
    c.none = p.splits > 1 && w.split >= chunks;
    c.c0 = base + static_cast<int32_t>((w.split * each + min(w.split, more)) * kStep);
    c.c1 = max(c.c0, min(c.c0 + static_cast<int32_t>((each + (w.split < more)) * kStep), hi));
    return c;
}

// Without a chunk: the join gives these rows no weight.
__device__ __forceinline__ void no_chunk(const TreeParams &p, const Work &w, const Rows &rows) {
    for (uint32_t i = threadIdx.x; i < rows.rows; i += blockDim.x) {
        float *to = p.stats + 2 * (out_row(p, w, rows, i) + w.chunk * p.nodes * p.q_heads);
        to[0] = -INFINITY;
        to[1] = 0;
    }
}

__device__ __forceinline__ uint32_t pages_of(const TreeParams &p, const Chunk &c) {
    return c.c1 > c.c0 ? (static_cast<uint32_t>(c.c1 - 1) >> p.page_shift) - (static_cast<uint32_t>(c.c0) >> p.page_shift) + 1 : 0;
}

// The chunk's pages into LDS, -1 for those that mask; whether there is one.
__device__ __forceinline__ int32_t load_pages(const TreeParams &p, const Work &w, const Chunk &c, int32_t *s_page) {
    const uint32_t n = pages_of(p, c);
    const int32_t *table = p.table + w.b * p.table_stride + (static_cast<uint32_t>(c.c0) >> p.page_shift);
    int32_t masked = 0;
    for (uint32_t i = threadIdx.x; i < n; i += blockDim.x) {
        const int32_t e = table[i];
        const bool ok = e >= 0 && static_cast<uint64_t>(e) < p.n_pages;
        s_page[i] = ok ? e : -1;
        masked |= !ok;
    }
    return masked;
}

// Whether positions p0..p0 + n - 1 have to be looked at one by one.
__device__ __forceinline__ bool masked_at(const Chunk &c, bool holes, int32_t p0, uint32_t n) {
    return holes || p0 < c.lo_max || p0 + static_cast<int32_t>(n) > min(c.all_hi, c.c1);
}

// Of a lane's eight positions, 4 q + 0..3 of each half of a step, those that lie
// in the chunk, past every start and in pages of the cache.
__device__ __forceinline__ uint32_t positions_there(const TreeParams &p, const Chunk &c, const int32_t *s_page, int32_t p0, uint32_t q) {
    const uint32_t first = static_cast<uint32_t>(c.c0) >> p.page_shift;
    uint32_t there = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int32_t pos0 = p0 + 16 * t + 4 * static_cast<int32_t>(q);
        const bool page = s_page[(static_cast<uint32_t>(min(pos0, c.c1 - 1)) >> p.page_shift) - first] >= 0;
        there |= page ? (bits_between(c.lo - pos0, c.c1 - pos0) & 15u) << (4 * t) : 0u;
    }
    return there;
}

// Those that a row reads.
__device__ __forceinline__ uint32_t positions_read(const TreeParams &p, const Work &w, const Rows &rows, const Row &row, const uint64_t *first, int32_t p0,
                                                   uint32_t q) {
    uint32_t live = bits_between(row.start - p0, rows.len - p0);
    const int32_t a0 = p0 - rows.len;  // the node at p0
    if (a0 + static_cast<int32_t>(kStep) > 0) {
        if (!p.mask) {
            live |= bits_between(-a0, min(row.node + 1, rows.count) - a0);
        } else if (a0 < rows.count) {
            const uint32_t from = static_cast<uint32_t>(max(a0, 0));
            const uint32_t at = from / 64, shift = from % 64;
            uint64_t m = *first;
            if (p.nodes > 64) {
                const int64_t *words = p.mask + w.b * p.mask_batch + static_cast<uint32_t>(row.node) * p.mask_node;
                m = static_cast<uint64_t>(words[at]) >> shift;
                if (shift > 32 && 64 * (at + 1) < p.nodes) m |= static_cast<uint64_t>(words[at + 1]) << (64 - shift);
            } else {
                m >>= shift;
            }
            live |= static_cast<uint32_t>(a0 < 0 ? m << -a0 : m) & bits_between(-a0, rows.count - a0);
        }
    }
    return ((live >> (4 * q)) & 15u) | (((live >> (16 + 4 * q)) & 15u) << 4);
}

// V rows of a step, a lane's piece of each of its eight positions (of one page
// for each half: pages hold multiples of 8).
template <int kWords>
struct Piece {
    typedef uint32_t Value __attribute__((ext_vector_type(kWords)));
    typedef Value InMemory __attribute__((aligned(4)));
};

template <int kWords, class Values>
__device__ __forceinline__ void load_v_rows(const TreeParams &p, const Chunk &c, const int32_t *s_page, const uint8_t *vb, int32_t p0,
                                            uint32_t r, uint32_t q, Values &vr) {
    const uint32_t first = static_cast<uint32_t>(c.c0) >> p.page_shift, in_page = (1u << p.page_shift) - 1;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int32_t pos0 = p0 + 16 * t + 4 * static_cast<int32_t>(q);
        const int32_t page = s_page[(static_cast<uint32_t>(min(pos0, c.c1 - 1)) >> p.page_shift) - first];
        const uint8_t *at_page = vb + static_cast<uint64_t>(max(page, 0)) * p.v.page + r * (kWords * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t at = static_cast<uint32_t>(min(pos0 + i, c.c1 - 1));
            vr[4 * t + i] = *reinterpret_cast<const typename Piece<kWords>::InMemory *>(at_page + uint64_t{at & in_page} * p.v.row);
        }
    }
}

// The running softmax of a lane's row over its wave's positions: weights are
// exp2(s scale - ref), where ref follows the maximum (less the lift) as soon as it is
// left more than kSlack behind.
template <int kPiece, bool kE4M3>
struct Running {
    static constexpr float kBelow = kE4M3 ? kLift : 0.0f;
    float ref = -INFINITY, sum = 0;  // sum: over this lane's positions
    f4 acc[kPiece] = {};

    // Takes the largest of some scores (of this lane's; scale > 0) into the reference.
    __device__ __forceinline__ void follow(float top, float scale) {
        const bool behind = top > -INFINITY && !(top * scale <= ref + (kSlack + kBelow));
        if (__builtin_expect(__any(behind), 0)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float to = top > -INFINITY ? fmaxf(ref, top * scale - kBelow) : ref;
            const float fade = to == ref ? 1.0f : exp2_(ref - to);
            ref = to;
            sum *= fade;
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[j][c] *= fade;
        }
    }

    // Turns a step's scores, -infinity where a position is masked, into weights.
    __device__ __forceinline__ void weights(const f4 (&s)[2], float scale, float (&w)[8]) {
        const float from = ref == -INFINITY ? 0.0f : ref;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = exp2_(fmaf(s[i / 4][i & 3], scale, -from));
            sum += w[i];
        }
    }
};

__device__ __forceinline__ float largest(const f4 (&s)[2], float top) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, s[i / 4][i & 3]);
    return top;
}

// Scores of positions that are not read become -infinity.
__device__ __forceinline__ void mask_scores(f4 (&s)[2], uint32_t live) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i / 4][i & 3] = live >> i & 1u ? s[i / 4][i & 3] : -INFINITY;
}

// Weights as the product with V takes them: FP16 beside FP16 values (from E4M3),
// or two parts of BF16, the second of which is held to at least `least`: where
// nothing is masked, above zero, so that an infinity in V stays what it is.
template <bool kE4M3>
__device__ __forceinline__ void pack_weights(const float (&w)[8], uint32_t least, v4u &high, v4u &low) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kE4M3) {
            high[i] = pack2h(w[2 * i], w[2 * i + 1]);
        } else {
            high[i] = cut2(w[2 * i], w[2 * i + 1]);
            low[i] = at_least2(pack2b(w[2 * i] - __builtin_bit_cast(float, high[i] << 16),
                                      w[2 * i + 1] - __builtin_bit_cast(float, high[i] & 0xFFFF0000u)),
                               least);
        }
    }
}

template <bool kE4M3>
__device__ __forceinline__ f4 product(const v4u &vt, const v4u &high, const v4u &low, f4 o) {
    if (kE4M3) return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, vt), __builtin_bit_cast(h8, high), o, 0, 0, 0);
    o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, vt), __builtin_bit_cast(bf8, high), o, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, vt), __builtin_bit_cast(bf8, low), o, 0, 0, 0);
}

// Four 16-bit values of a row from each of four lanes in four: lane r of 16 gives
// those of row r / 4 at `at`, and gets value r % 4 of the rows r / 4 gave, of all four.
__device__ __forceinline__ v2u read_transposed(const uint8_t *at) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4 Lds;
    return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds *)(at)));
}

// The same of 8-bit values: eight of a row from each of two lanes, of eight rows.
__device__ __forceinline__ v2u read_transposed8(const uint8_t *at) {
    typedef int i2 __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(3))) i2 Lds;
    return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr8_b64_v2i32((Lds *)(at)));
}

// Values j and j + 1 of a lane's eight rows, each as an operand: V^T's rows.
__device__ __forceinline__ void transpose(const uint32_t (&pair)[8], v4u (&vt)[2]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t sel = e ? 0x07060302u : 0x05040100u;
        vt[e] = v4u{__builtin_amdgcn_perm(pair[1], pair[0], sel), __builtin_amdgcn_perm(pair[3], pair[2], sel),
                    __builtin_amdgcn_perm(pair[5], pair[4], sel), __builtin_amdgcn_perm(pair[7], pair[6], sel)};
    }
}

// What is no finite number in V is left out of a masked step's product, as 0
// times it would reach rows that do not read it.  If there was any it is added
// after all steps: a product of ones counts for each row how many of those that it
// reads are infinities of either sign or NaN.  kStrided: a lane's values of V^T's
// tile j are those of d = 16 j + r, otherwise of d = r kDim / 16 + j.
template <int kDim, bool kE4M3, int kTiles, bool kStrided>
__device__ __forceinline__ void add_counts(const TreeParams &p, const Work &work, const Rows &rows, const Row (&row)[kTiles], const uint64_t *s_first,
                                           const uint8_t *vb, const int32_t *s_page, const Chunk &c, int32_t p0, Running<kDim / 16, kE4M3> (&run)[kTiles]) {
    constexpr int kPiece = kDim / 16;
    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, q = lane >> 4;
    const uint32_t first = static_cast<uint32_t>(c.c0) >> p.page_shift, in_page = (1u << p.page_shift) - 1;
    const uint32_t there = positions_there(p, c, s_page, p0, q);
    v4u ones[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const uint32_t live = positions_read(p, work, rows, row[t], &s_first[16 * t + r], p0, q) & there;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            ones[t][i] = (live >> (2 * i) & 1u ? 0x3F80u : 0u) | (live >> (2 * i + 1) & 1u ? 0x3F800000u : 0u);
    }
    const uint8_t *at[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t pos = static_cast<uint32_t>(min(p0 + 16 * (i / 4) + 4 * static_cast<int32_t>(q) + (i & 3), c.c1 - 1));
        at[i] = vb + static_cast<uint64_t>(max(s_page[(pos >> p.page_shift) - first], 0)) * p.v.page + uint64_t{pos & in_page} * p.v.row;
    }
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
        const uint32_t d = kStrided ? 16 * j + r : r * kPiece + j;
        v4u kinds;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            kinds[i] = (there >> (2 * i) & 1u ? kind_at<kE4M3>(at[2 * i], d) : 0u) | (there >> (2 * i + 1) & 1u ? kind_at<kE4M3>(at[2 * i + 1], d) : 0u) << 16;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const f4 n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, kinds), __builtin_bit_cast(bf8, ones[t]), f4{}, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k) run[t].acc[j][k] += of_counts(n[k]);
        }
    }
}

constexpr int waves_for(int dim) { return dim == 64 ? 3 : dim == 128 ? 2 : 1; }

// Few rows: the waves of a workgroup have all of a tile's rows (up to 32) each
// and take the chunk's steps in turn, keys and values coming straight from
// memory, each once; they join in LDS.  No barrier stands in the loop, and a step's
// loads are on their way while the one before is computed.  Bound by HBM and, for short
// sequences, by start and end: 16 sequences of 4,096 with 8 nodes of 32 heads (268 MB)
// 59 us, 4.6 TB/s, E4M3 34, 4.0; 1 x 8,192 with 8 nodes 19 us.  Through LDS (below) those
// take 64, 39 and 21.  Heads of 256 take one tile of rows: two need more registers than there are.
template <int kDim, bool kE4M3, int kTiles>
__global__ void __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(waves_for(kDim))))
tree_few_kernel(TreeParams p) {
    constexpr int kPiece = kDim / 16;              // values of a V row in a lane; tiles of out^T
    constexpr int kKChunks = kDim / 32;            // matrix instructions over d
    constexpr int kKLoads = kE4M3 ? kDim / 64 : kKChunks;  // 16-byte loads of a K row in a lane
    constexpr int kVWords = kPiece * (kE4M3 ? 1 : 2) / 4;  // dwords of a V piece
    constexpr uint32_t kRows = 16 * kTiles;
    __shared__ int32_t s_page[kChunkPages];
    __shared__ uint64_t s_first[kRows];
    __shared__ float s_stat[kWaves][2][16];
    __shared__ __attribute__((aligned(16))) float s_out[kWaves][16][kDim + kPad];

    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Work work = work_of(p);
    if (work.none) return;
    const Rows rows = rows_of(p, work, kRows);
    Row row[kTiles];
    int32_t lo = rows.len, lo_max = 0;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        row[t] = row_of(p, work, rows, 16 * t + r, &s_first[16 * t + r]);
        lo = row[t].have ? min(lo, row[t].start) : lo;
        lo_max = row[t].have ? max(lo_max, row[t].start) : lo_max;
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
    Chunk c = chunk_of(p, work, rows, lo, lo_max);
    if (c.none) {
        no_chunk(p, work, rows);
        return;
    }
    const int32_t end = c.c1;
    c.c1 = min(end, c.c0 + static_cast<int32_t>(kMaxChunk));
    const int32_t masked_pages = load_pages(p, work, c, s_page);

    // Q^T: row r of each tile, d in the order in which K's loads give them.  A
    // negative scale turns q around, so that the largest product is the largest
    // score, and one of zero makes q zero.
    const float signed_scale = kE4M3 ? p.scale * p.k.scale[work.h] : p.scale;
    const float scale = signed_scale == 0 ? 1.0f : fabsf(signed_scale);
    const uint32_t turned = signed_scale < 0 ? 0x80008000u : 0;
    bf8 qf[kTiles][kKChunks];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const uint32_t n = min(rows.row0 + 16 * t + r, p.nodes * p.group - 1);
        const uint16_t *qp = p.q + work.b * p.q_batch + static_cast<uint32_t>(row[t].node) * p.q_node +
                             (work.h * p.group + (n - static_cast<uint32_t>(row[t].node) * p.group)) * p.q_head;
#pragma unroll
        for (int i = 0; i < kKChunks; ++i) {
            const uint32_t d = kE4M3 ? 64 * (i / 2) + 16 * q + 8 * (i & 1) : 32 * i + 8 * q;
            v4u w = row[t].have && signed_scale != 0 ? load8(qp + d) : v4u{0, 0, 0, 0};
            w ^= turned;
            qf[t][i] = __builtin_bit_cast(bf8, w);
        }
    }
    const uint8_t *kb = p.k.base + work.h * p.k.head, *vb = p.v.base + work.h * p.v.head;
    const uint32_t in_page = (1u << p.page_shift) - 1;
    uint32_t first = static_cast<uint32_t>(c.c0) >> p.page_shift;
    bool holes = __syncthreads_or(masked_pages);  // and the pages are there

    // K rows of a step: lane r has position r of each half
    v4u kr[2][kKLoads];
    auto load_k = [&](int32_t p0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t pos = static_cast<uint32_t>(min(p0 + 16 * t + static_cast<int32_t>(r), c.c1 - 1));
            const int32_t page = max(s_page[(pos >> p.page_shift) - first], 0);
            const uint8_t *at = kb + static_cast<uint64_t>(page) * p.k.page + uint64_t{pos & in_page} * p.k.row + 16 * q;
#pragma unroll
            for (int i = 0; i < kKLoads; ++i) kr[t][i] = *reinterpret_cast<const v4u *>(at + 64 * i);
        }
    };
    typename Piece<kVWords>::Value vr[8];
    auto load_v = [&](int32_t p0) { load_v_rows<kVWords>(p, c, s_page, vb, p0, r, q, vr); };

    Running<kPiece, kE4M3> run[kTiles];
    uint32_t odd = 0;  // whether some value of V was left out of masked steps
    auto step = [&](int32_t p0, int32_t next) {
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

        const bool masked = masked_at(c, holes, p0, kStep);
        if (__builtin_expect(masked, false)) {
            const uint32_t there = positions_there(p, c, s_page, p0, q);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) mask_scores(s[t], positions_read(p, work, rows, row[t], &s_first[16 * t + r], p0, q) & there);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!(there >> i & 1u)) vr[i] = 0;
#pragma unroll
                for (int w = 0; w < kVWords; ++w) {
                    const uint32_t n = not_finite<kE4M3>(vr[i][w]);
                    odd |= n;
                    vr[i][w] &= ~n;
                }
            }
        }
        v4u high[kTiles], low[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            float w[8];
            run[t].follow(largest(s[t], -INFINITY), scale);
            run[t].weights(s[t], scale, w);
            pack_weights<kE4M3>(w, masked ? 0u : kLeastPart, high[t], low[t]);
        }
#pragma unroll
        for (int j = 0; j < kPiece; j += 2) {
            uint32_t pair[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (kE4M3)
                    pair[i] = j & 2 ? half_from_e4m3<true>(vr[i][j / 4]) : half_from_e4m3<false>(vr[i][j / 4]);
                else
                    pair[i] = vr[i][kE4M3 ? 0 : j / 2];
            }
            v4u vt[2];
            transpose(pair, vt);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int t = 0; t < kTiles; ++t) run[t].acc[j + e] = product<kE4M3>(vt[e], high[t], low[t], run[t].acc[j + e]);
        }
        load_v(next);
    };
    for (;;) {  // once for the pages that LDS holds
        const int32_t wave0 = c.c0 + static_cast<int32_t>(wave * kStep);
        if (wave0 < c.c1) {
            load_k(wave0);
            load_v(wave0);
            // the last step loads its chunk's last row in vain
            for (int32_t p0 = wave0; p0 < c.c1; p0 += kWaves * kStep) step(p0, p0 + kWaves * kStep);
            if (__builtin_expect(__any(odd != 0), 0))
                for (int32_t p0 = wave0; p0 < c.c1; p0 += kWaves * kStep)
                    if (masked_at(c, holes, p0, kStep)) add_counts<kDim, kE4M3, kTiles, false>(p, work, rows, row, s_first, vb, s_page, c, p0, run);
            odd = 0;
        }
        if (c.c1 >= end) break;
        __syncthreads();
        c.c0 = c.c1;
        c.c1 = min(end, c.c0 + static_cast<int32_t>(kMaxChunk));
        first = static_cast<uint32_t>(c.c0) >> p.page_shift;
        holes = __syncthreads_or(load_pages(p, work, c, s_page));
    }

    // join the waves, a tile at a time
    const float v_scale = kE4M3 ? p.v.scale[work.h] : 1.0f;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        if (16u * t >= rows.rows) break;
        float sum = run[t].sum;
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (t) __syncthreads();  // the last tile has been read
        if (q == 0) {
            s_stat[wave][0][r] = run[t].ref;
            s_stat[wave][1][r] = sum;
        }
        // acc[j][c]: d = (4 q + c) * kPiece + j
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < kPiece; j += 4)
                *reinterpret_cast<f4 *>(&s_out[wave][r][(4 * q + k) * kPiece + j]) =
                    f4{run[t].acc[j][k], run[t].acc[j + 1][k], run[t].acc[j + 2][k], run[t].acc[j + 3][k]};
        __syncthreads();
        constexpr uint32_t kQuads = kDim / 4;
        for (uint32_t i = threadIdx.x; i < min(16u, rows.rows - 16 * t) * kQuads; i += 64 * kWaves) {
            const uint32_t g = i / kQuads, d = i % kQuads * 4;
            const bool there = static_cast<int32_t>((rows.row0 + 16 * t + g) / p.group) < rows.count;
            float top = -INFINITY;
#pragma unroll
            for (uint32_t k = 0; k < kWaves; ++k) top = fmaxf(top, s_stat[k][0][g]);
            const float from = top == -INFINITY ? 0.0f : top;
            float total = 0;
            f4 o = {};
#pragma unroll
            for (uint32_t k = 0; k < kWaves; ++k) {
                const float f = exp2_(s_stat[k][0][g] - from);
                total += s_stat[k][1][g] * f;
                o += *reinterpret_cast<const f4 *>(&s_out[k][g][d]) * f;
            }
            write_out<kDim>(p, work.chunk, out_row(p, work, rows, 16 * t + g), d, there, top, total, o * v_scale);
        }
    }
}

// Many rows: keys and values go through LDS, once for a workgroup, as they are
// stored, by loads that are stages ahead of their use.  kGroups of the waves share a
// wave's 16 kTiles rows and take a stage's steps in turn; they join in LDS.  A row's
// 16-byte pieces lie there in an order of its own, so that lanes that read a piece
// of different rows do not meet in a bank: K is read piece by piece of 16 rows, V
// across rows by the hardware's transposing reads, which give V^T.  E4M3 becomes
// BF16 (keys) and FP16 (values) in registers.
// A K or V row that comes straight from memory is read by each wave anew, at 64 bytes a
// cycle and compute unit: 64 rows would spend more time on that than on matrix
// instructions.  64 KiB of stages (two of BF16, four of E4M3) leave place for two
// workgroups, whose waves fill each other's waits.  Bound by the vector and the matrix unit,
// which overlap little: a step of 32 rows and 32 positions of 128 takes a SIMD about 1,800
// cycles, 768 of them matrix instructions.  8 x 32,768 with 16 nodes of 64 heads: BF16 257
// us (4.2 TB/s, 536 TFLOP/s), E4M3 178 (773 TFLOP/s); 1 x 8,192 with 64 nodes of 32 heads
// 32, of which start and end are about 10; chains of 509 over heads of 256 39 (the joins
// among them).
constexpr uint32_t kManyWaves = 4;

template <int kDim>
constexpr uint32_t kStagePositions = 8192 / kDim;

template <int kDim, bool kE4M3>
__device__ __forceinline__ uint32_t k_turn(uint32_t row) {
    constexpr uint32_t kPieces = kDim * (kE4M3 ? 1 : 2) / 16;
    return kPieces >= 16 ? row & 15u : kPieces == 8 ? row >> (kE4M3 ? 1 : 0) & 7u : row >> 2 & 3u;
}

template <int kDim, bool kE4M3>
__device__ __forceinline__ uint32_t v_turn(uint32_t row) {
    constexpr uint32_t kPieces = kDim * (kE4M3 ? 1 : 2) / 16;
    if (!kE4M3) return kPieces == 8 ? row & 6u : 2 * (row & 7u);
    return kPieces >= 16 ? (row & 7u) | (row >> 1 & 8u) : kPieces == 8 ? (row >> 1 & 3u) | (row >> 2 & 4u) : (row >> 2 & 1u) | (row >> 3 & 2u);
}

// 16 bytes for each lane, from its offset, into LDS next to each other from `to` on
// (uniform, like the base).  By hand: behind the builtin the compiler lets transposing
// reads of other arrays wait for it, too.  Nothing is returned to a register, and
// arrived() waits for what was loaded.  The place is an operand in m0, which the
// compiler sets and so knows the contents of.  m0 is there for a load into LDS one
// cycle after it is written, and a scalar register that the vector unit wrote five.
__device__ __forceinline__ void load_lds(const uint8_t *from, uint32_t offset, uint32_t to) {
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(to), "v"(offset), "s"(from) : "memory");
}

// The same from two bases.
__device__ __forceinline__ void load_lds(const uint8_t *from, const uint8_t *from2, bool second, uint32_t offset, uint32_t to) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(to), "v"((second ? from2 : from) + offset) : "memory");
}

__device__ __forceinline__ uint32_t place_of(uint8_t *stage) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)(stage)));
}

// Waits for this wave's loads but the last kAfter, those into LDS among them: a
// barrier alone does not (vmcnt; the other counters as they are).
template <int kAfter>
__device__ __forceinline__ void arrived() {
    static_assert(kAfter < 16, "four bits of the count");
    __builtin_amdgcn_s_waitcnt(0x0F70 | kAfter);
}

template <int kDim, bool kE4M3, int kTiles, uint32_t kGroups>
__global__ void __launch_bounds__(64 * kManyWaves, 2) tree_many_kernel(TreeParams p) {
    constexpr int kPiece = kDim / 16, kKChunks = kDim / 32;
    constexpr uint32_t kThreads = 64 * kManyWaves, kRows = 16 * kTiles * kManyWaves / kGroups, kStage = kStagePositions<kDim>;
    constexpr uint32_t kRowBytes = kDim * (kE4M3 ? 1 : 2), kPieces = kRowBytes / 16, kBytes = kStage * kRowBytes;  // of a stage's K, and V
    constexpr uint32_t kRing = kE4M3 ? 4 : 2;  // stages, 64 KiB
    static_assert(kStage % (kStep * kGroups) == 0 && kTiles * kPiece * 1024 <= 2 * kBytes * kRing / kManyWaves, "stages hold what the waves join");
    __shared__ int32_t s_page[kChunkPages];
    __shared__ uint64_t s_first[kRows];
    __shared__ int32_t s_reads[2][kManyWaves];
    __shared__ float s_stat[kManyWaves][kTiles][2][16];
    // K and V of each stage: arrays of their own, as the compiler waits for loads into
    // one before it reads from it
    __shared__ __attribute__((aligned(16))) uint8_t s_ring0[2 * kBytes], s_ring1[2 * kBytes];
    __shared__ __attribute__((aligned(16))) uint8_t s_ring2[kRing > 2 ? 2 * kBytes : 16], s_ring3[kRing > 2 ? 2 * kBytes : 16];

    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t group = wave % kGroups;
    const Work work = work_of(p);
    if (work.none) return;
    const Rows rows = rows_of(p, work, kRows);
    const uint32_t wave_row = wave / kGroups * 16 * kTiles;
    const bool active = wave_row < rows.rows;  // others fetch and wait
    Row row[kTiles];
    int32_t lo = rows.len, lo_max = 0;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        row[t] = row_of(p, work, rows, wave_row + 16 * t + r, &s_first[wave_row + 16 * t + r]);
        lo = row[t].have ? min(lo, row[t].start) : lo;
        lo_max = row[t].have ? max(lo_max, row[t].start) : lo_max;
    }
    if (p.starts) {
#pragma unroll
        for (int i = 1; i < 16; i <<= 1) {
            lo = min(lo, __shfl_xor(lo, i));
            lo_max = max(lo_max, __shfl_xor(lo_max, i));
        }
        if (lane == 0) {
            s_reads[0][wave] = lo;
            s_reads[1][wave] = lo_max;
        }
        __syncthreads();
        lo = rows.len;
        lo_max = 0;
#pragma unroll
        for (uint32_t w = 0; w < kManyWaves; ++w) {
            lo = min(lo, s_reads[0][w]);
            lo_max = max(lo_max, s_reads[1][w]);
        }
        lo = __builtin_amdgcn_readfirstlane(lo);
        lo_max = __builtin_amdgcn_readfirstlane(lo_max);
    } else {
        lo = lo_max = 0;
    }
    Chunk c = chunk_of(p, work, rows, lo, lo_max);
    if (c.none) {
        no_chunk(p, work, rows);
        return;
    }
    const int32_t end = c.c1;
    c.c1 = min(end, c.c0 + static_cast<int32_t>(kMaxChunk));
    const int32_t masked_pages = load_pages(p, work, c, s_page);

    const float signed_scale = kE4M3 ? p.scale * p.k.scale[work.h] : p.scale;
    const float scale = signed_scale == 0 ? 1.0f : fabsf(signed_scale);
    v4u qw[kTiles][kKChunks];  // on its way until the first stage is
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const uint32_t n = min(rows.row0 + wave_row + 16 * t + r, p.nodes * p.group - 1);
        const uint16_t *qp = p.q + work.b * p.q_batch + static_cast<uint32_t>(row[t].node) * p.q_node +
                             (work.h * p.group + (n - static_cast<uint32_t>(row[t].node) * p.group)) * p.q_head;
#pragma unroll
        for (int i = 0; i < kKChunks; ++i) qw[t][i] = load8(qp + (kE4M3 ? 64 * (i / 2) + 16 * q + 8 * (i & 1) : 32 * i + 8 * q));
    }
    const uint8_t *kb = p.k.base + work.h * p.k.head, *vb = p.v.base + work.h * p.v.head;
    const uint32_t in_page = (1u << p.page_shift) - 1;
    uint32_t first = static_cast<uint32_t>(c.c0) >> p.page_shift;
    bool holes = __syncthreads_or(masked_pages);  // and the pages are there

    uint32_t odd = 0;  // whether some value of V was left out of masked stages
    auto clean = [&](int32_t pos, v4u &v) {  // nothing of V where no row reads, nothing that is no finite number
        const bool there = pos >= c.lo && pos < c.c1 && s_page[(static_cast<uint32_t>(min(pos, c.c1 - 1)) >> p.page_shift) - first] >= 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (!there) v[w] = 0;
            const uint32_t n = not_finite<kE4M3>(v[w]);
            odd |= n;
            v[w] &= ~n;
        }
    };
    // Loads of a stage into LDS, a wave's next to each other: lane i's piece goes to
    // place i.  Rows of one load lie in one page each eight: where such eight begin
    // is the same for all lanes, and a lane's own part of an address stays what it is.
    constexpr uint32_t kLoadRows = 64 / kPieces, kFetches = kStage / (kLoadRows * kManyWaves);  // rows of a load; loads of K
    constexpr uint32_t kEights = kLoadRows > 8 ? 2 : 1;
    struct Fetch {
        const uint8_t *k[kFetches][kEights], *v[kFetches][kEights];
        uint32_t to;
    };
    auto find = [&](int32_t p0, uint32_t to) {
        uint32_t at[kFetches][kEights];
        int32_t page[kFetches][kEights];
#pragma unroll
        for (uint32_t i = 0; i < kFetches; ++i)
#pragma unroll
            for (uint32_t e = 0; e < kEights; ++e) {
                // past the end the last rows again
                at[i][e] = static_cast<uint32_t>(min(p0 + static_cast<int32_t>(((i * kManyWaves + wave) * kLoadRows & ~7u) + 8 * e), (c.c1 - 1) & ~7));
                page[i][e] = s_page[(at[i][e] >> p.page_shift) - first];
            }
        __builtin_amdgcn_sched_barrier(0);  // all of them on their way before the first is waited for
        Fetch f;
        f.to = to;
#pragma unroll
        for (uint32_t i = 0; i < kFetches; ++i)
#pragma unroll
            for (uint32_t e = 0; e < kEights; ++e) {
                const uint32_t n = static_cast<uint32_t>(max(__builtin_amdgcn_readfirstlane(page[i][e]), 0)), in = at[i][e] & in_page;
                f.k[i][e] = kb + n * p.k.page + in * p.k.row;
                f.v[i][e] = vb + n * p.v.page + in * p.v.row;
            }
        return f;
    };
    uint32_t from_k[kFetches], from_v[kFetches];  // of a lane, from where its eight rows begin
#pragma unroll
    for (uint32_t i = 0; i < kFetches; ++i) {
        const uint32_t row = (i * kManyWaves + wave) * kLoadRows + lane / kPieces, place = lane % kPieces;
        from_k[i] = row % 8 * static_cast<uint32_t>(p.k.row) + 16 * (place ^ k_turn<kDim, kE4M3>(row));
        from_v[i] = row % 8 * static_cast<uint32_t>(p.v.row) + 16 * (place ^ v_turn<kDim, kE4M3>(row));
    }
    auto fetch = [&](const Fetch &f, uint32_t i) {
        const uint32_t to = f.to + (i * kManyWaves + wave) * kLoadRows * kRowBytes;
        if constexpr (kEights > 1) {
            const bool second = lane >= 8 * kPieces;
            load_lds(f.k[i][0], f.k[i][1], second, from_k[i], to);
            load_lds(f.v[i][0], f.v[i][1], second, from_v[i], to + kBytes);
        } else {
            load_lds(f.k[i][0], from_k[i], to);
            load_lds(f.v[i][0], from_v[i], to + kBytes);
        }
    };
    auto fetch_all = [&](const Fetch &f) {
#pragma unroll
        for (uint32_t i = 0; i < kFetches; ++i) fetch(f, i);
    };
    uint8_t *const ring[4] = {s_ring0, s_ring1, s_ring2, s_ring3};
    const uint32_t places[4] = {place_of(s_ring0), place_of(s_ring1), place_of(s_ring2), place_of(s_ring3)};
    auto fetch_first = [&] {
#pragma unroll
        for (uint32_t i = 0; i + 1 < kRing; ++i) fetch_all(find(c.c0 + static_cast<int32_t>(i * kStage), places[i]));
    };
    auto clean_stage = [&](int32_t p0, uint8_t *stage) {  // what has arrived
        constexpr uint32_t kEach = kStage * kPieces / kThreads;
        v4u *at = reinterpret_cast<v4u *>(stage + kBytes) + threadIdx.x;
        v4u v[kEach];
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i) v[i] = at[i * kThreads];
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i) {
            clean(p0 + static_cast<int32_t>((i * kThreads + threadIdx.x) / kPieces), v[i]);
            at[i * kThreads] = v[i];
        }
    };

    if (c.c0 < c.c1) fetch_first();
    bf8 qf[kTiles][kKChunks];
    const uint32_t turned = signed_scale < 0 ? 0x80008000u : 0;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < kKChunks; ++i) {
            const v4u w = row[t].have && signed_scale != 0 ? qw[t][i] : v4u{0, 0, 0, 0};
            qf[t][i] = __builtin_bit_cast(bf8, w ^ turned);
        }

    Running<kPiece, kE4M3> run[kTiles];
    constexpr int kSteps = kStage / (kStep * kGroups);  // of a wave in a stage
    // Where a lane reads in a stage: rows 16 and 32 further on take their pieces in the
    // same order, so that steps and stages are constants of the instructions.  Unknown
    // to the compiler, which would keep these places for each stage.
    constexpr int kKReads = kE4M3 ? kKChunks / 2 : kKChunks;  // 16 bytes of a K row each
    uint32_t k_at[kKReads], v_at[kPiece];
#pragma unroll
    for (int i = 0; i < kKReads; ++i) {
        k_at[i] = (group * kStep + r) * kRowBytes + 16 * ((4 * i + q) ^ k_turn<kDim, kE4M3>(r));
        asm("" : "+v"(k_at[i]));
    }
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
        const uint32_t at = kE4M3 ? 16 * (r / 8) + 4 * q + (r / 2 & 3u) : 4 * q + r / 4;
        v_at[j] = kBytes + (group * kStep + at) * kRowBytes + 8 * (r & 1u) +
                  16 * ((kE4M3 ? j : 2 * j + (r & 3u) / 2) ^ v_turn<kDim, kE4M3>(at));
        asm("" : "+v"(v_at[j]));
    }
    // A wave's steps of a stage, positions p0 and on: all scores first, then a step's
    // weights beside the product of those before.  Loads of a later stage go out
    // between them, as a compute unit takes 64 bytes of them in a cycle.
    auto steps = [&](int32_t p0, const uint8_t *stage, bool masked, const Fetch &later) {
        constexpr int kPlaces = 2 * kSteps + kSteps * (kPiece / 4);
        const auto go_on = [&](int place) {
#pragma unroll
            for (uint32_t i = 0; i < kFetches; ++i)
                if (place == static_cast<int>(i * kPlaces / kFetches)) fetch(later, i);
        };
        f4 s[kSteps][kTiles][2] = {};
        // reads from LDS stay a group ahead of what takes them: nothing of them is
        // moved over these places, all else is
        const auto keep_reads = [] { __builtin_amdgcn_sched_barrier(0x7F); };
        v4u kf[2][kKReads];
        const auto read_k = [&](int n) {
#pragma unroll
            for (int i = 0; i < kKReads; ++i)
                kf[n & 1][i] = *reinterpret_cast<const v4u *>(stage + k_at[i] + (n / 2 * kGroups * kStep + 16 * (n & 1)) * kRowBytes);
        };
        read_k(0);
#pragma unroll
        for (int n = 0; n < 2 * kSteps; ++n) {
            if (n + 1 < 2 * kSteps) read_k(n + 1);
            keep_reads();
            go_on(n);
#pragma unroll
            for (int i = 0; i < kKChunks; ++i) {
                v4u kw = kf[n & 1][kE4M3 ? i / 2 : i];
                if (kE4M3) kw = i & 1 ? from_e4m3x8(kw.z, kw.w) : from_e4m3x8(kw.x, kw.y);
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
                    s[n / 2][t][n & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, kw), qf[t][i], s[n / 2][t][n & 1], 0, 0, 0);
            }
        }
        constexpr int kBlock = 4, kBlocks = kPiece / kBlock;  // of V^T's tiles
        v2u vt[2][kBlock][kE4M3 ? 1 : 2];
        const auto read_v = [&](int n) {
            const uint8_t *from = stage + n / kBlocks * kGroups * kStep * kRowBytes;
#pragma unroll
            for (int j = 0; j < kBlock; ++j) {
                const uint32_t at = v_at[n % kBlocks * kBlock + j];
                if (kE4M3) {
                    vt[n & 1][j][0] = read_transposed8(from + at);
                } else {
#pragma unroll
                    for (int u = 0; u < 2; ++u) vt[n & 1][j][kE4M3 ? 0 : u] = read_transposed(from + at + 16 * u * kRowBytes);
                }
            }
        };
        read_v(0);
        keep_reads();
        if (__builtin_expect(masked, false)) {
#pragma unroll
            for (int n = 0; n < kSteps; ++n) {
                const int32_t at = p0 + static_cast<int32_t>((n * kGroups + group) * kStep);
                const uint32_t there = positions_there(p, c, s_page, at, q);
#pragma unroll
                for (int t = 0; t < kTiles; ++t) mask_scores(s[n][t], positions_read(p, work, rows, row[t], &s_first[wave_row + 16 * t + r], at, q) & there);
            }
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < kSteps; ++n) top = largest(s[n][t], top);
            run[t].follow(top, scale);
        }
        const uint32_t least = masked ? 0u : kLeastPart;
#pragma unroll
        for (int n = 0; n < kSteps; ++n) {
            v4u high[kTiles], low[kTiles];
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                float w[8];
                run[t].weights(s[n][t], scale, w);
                pack_weights<kE4M3>(w, least, high[t], low[t]);
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int at = n * kBlocks + b;
                if (at + 1 < kSteps * kBlocks) read_v(at + 1);
                keep_reads();
                go_on(2 * kSteps + at);
#pragma unroll
                for (int j = 0; j < kBlock; ++j) {
                    const v2u x = vt[at & 1][j][0], y = vt[at & 1][j][kE4M3 ? 0 : 1];
                    const v4u v = kE4M3 ? v4u{half_from_e4m3<false>(x.x), half_from_e4m3<true>(x.x), half_from_e4m3<false>(x.y), half_from_e4m3<true>(x.y)}
                                        : v4u{x.x, x.y, y.x, y.y};
#pragma unroll
                    for (int t = 0; t < kTiles; ++t)
                        run[t].acc[b * kBlock + j] = product<kE4M3>(v, high[t], low[t], run[t].acc[b * kBlock + j]);
                }
            }
        }
    };
    while (c.c0 < c.c1) {  // once for the pages that LDS holds
        arrived<2 * kFetches * (kRing - 2)>();
        __syncthreads();
        const auto turn = [&](int32_t p0, uint32_t n) {  // a stage, number n of the ring
            const bool masked = masked_at(c, holes, p0, kStage);
            if (__builtin_expect(masked, false)) {
                clean_stage(p0, ring[n]);
                __syncthreads();
            }
            const Fetch later = find(p0 + static_cast<int32_t>((kRing - 1) * kStage), places[(n + kRing - 1) % kRing]);
            if (active)
                steps(p0, ring[n], masked, later);
            else
                fetch_all(later);
            arrived<2 * kFetches * (kRing - 2)>();
            __syncthreads();
        };
        for (int32_t p0 = c.c0; p0 < c.c1; p0 += kRing * kStage) {
#pragma unroll
            for (uint32_t n = 0; n < kRing; ++n) {
                const int32_t at = p0 + static_cast<int32_t>(n * kStage);
                if (at < c.c1) turn(at, n);
            }
        }
        arrived<0>();  // what was fetched past the end
        if (__builtin_expect(__syncthreads_or(odd != 0), 0))
            for (int32_t p0 = c.c0; p0 < c.c1; p0 += kStage)
                if (masked_at(c, holes, p0, kStage))
                    for (uint32_t at = kStep * group; at < kStage && p0 + static_cast<int32_t>(at) < c.c1; at += kStep * kGroups)
                        add_counts<kDim, kE4M3, kTiles, true>(p, work, rows, row, s_first + wave_row, vb, s_page, c, p0 + static_cast<int32_t>(at), run);
        if (c.c1 >= end) break;
        __syncthreads();
        odd = 0;
        c.c0 = c.c1;
        c.c1 = min(end, c.c0 + static_cast<int32_t>(kMaxChunk));
        first = static_cast<uint32_t>(c.c0) >> p.page_shift;
        holes = __syncthreads_or(load_pages(p, work, c, s_page));
        fetch_first();
    }

    const float v_scale = kE4M3 ? p.v.scale[work.h] : 1.0f;
    // the stages hold the waves' parts
    const auto part = [&](uint32_t g, int t, int j) -> f4 & {
        constexpr uint32_t kPer = kManyWaves / kRing;  // waves to a stage
        const uint32_t w = wave / kGroups * kGroups + g, n = w / kPer;
        return reinterpret_cast<f4 *>(n == 0 ? s_ring0 : n == 1 ? s_ring1 : n == 2 ? s_ring2 : s_ring3)[((w % kPer * kTiles + t) * kPiece + j) * 64 + lane];
    };
    if (kGroups > 1) {
        // every wave of a row group puts what it has side by side, and takes a share of all
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            float sum = run[t].sum;
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (q == 0) {
                s_stat[wave][t][0][r] = run[t].ref;
                s_stat[wave][t][1][r] = sum;
            }
#pragma unroll
            for (int j = 0; j < kPiece; ++j) part(group, t, j) = run[t].acc[j];
        }
        __syncthreads();
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const uint32_t i = wave_row + 16 * t + r;
        if (i >= rows.rows) continue;
        const uint64_t to = out_row(p, work, rows, i);
        float top = run[t].ref, total = 0, fade[kGroups];
        if (kGroups == 1) {
            total = run[t].sum;
            total += __shfl_xor(total, 16);
            total += __shfl_xor(total, 32);
        } else {
            const uint32_t wave0 = wave / kGroups * kGroups;
            top = -INFINITY;
#pragma unroll
            for (uint32_t g = 0; g < kGroups; ++g) top = fmaxf(top, s_stat[wave0 + g][t][0][r]);
            const float from = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (uint32_t g = 0; g < kGroups; ++g) {
                fade[g] = exp2_(s_stat[wave0 + g][t][0][r] - from);
                total += s_stat[wave0 + g][t][1][r] * fade[g];
            }
        }
        // acc[j][k]: d = 16 j + 4 q + k
#pragma unroll
        for (int n = 0; n < kPiece / static_cast<int>(kGroups); ++n) {
            const int j = n * kGroups;
            f4 o = run[t].acc[j];
            if (kGroups > 1) {
                o = f4{};
#pragma unroll
                for (uint32_t g = 0; g < kGroups; ++g) o += part(g, t, j + static_cast<int>(group)) * fade[g];
            }
            write_out<kDim>(p, work.chunk, to, 16 * (j + (kGroups > 1 ? group : 0)) + 4 * q, row[t].have, top, total, o * v_scale);
        }
    }
}

// Joins the chunks: kDim / 4 lanes, four values each, for every `share`-th chunk of
// a row (a power of two); LDS joins those.  Bound by latency: a lane has four
// chunks' values on their way.  About 5 us behind 1 x 8,192 with 64 nodes (16 chunks);
// with one lane for all chunks of a row, one after the other, 1 x 8,192 with 8 nodes (64
// chunks) took 53 us in place of 20.
constexpr uint32_t kJoinThreads = 256;

template <int kDim>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(TreeParams p, uint64_t rows, uint32_t share) {
    constexpr uint32_t kQuads = kDim / 4, kAhead = 4;
    __shared__ f4 s_part[kJoinThreads];
    __shared__ v2f s_stat[kJoinThreads];
    const uint32_t d = threadIdx.x % kQuads, group = threadIdx.x / kQuads % share;
    const uint64_t row = uint64_t{blockIdx.x} * (kJoinThreads / kQuads / share) + threadIdx.x / (kQuads * share);
    const uint32_t per = p.nodes * p.q_heads, b = static_cast<uint32_t>(row) / per;
    float top = -INFINITY, total = 0;
    f4 o = {};
    if (row < rows) {
        const uint32_t first = p.own ? p.own[2 * b] : b * p.splits, chunks = p.own ? p.own[2 * b + 1] : p.splits;
        const uint64_t row0 = uint64_t{first} * per + (static_cast<uint32_t>(row) - b * per);
        const v2f *stats = reinterpret_cast<const v2f *>(p.stats) + row0;
        const f4 *part = reinterpret_cast<const f4 *>(p.part + row0 * kDim) + d;
        for (uint32_t i0 = group; i0 < chunks; i0 += kAhead * share) {
            v2f s[kAhead];
            f4 v[kAhead];
            float most = top;
#pragma unroll
            for (uint32_t a = 0; a < kAhead; ++a) {
                const uint32_t i = i0 + a * share;
                s[a] = v2f{-INFINITY, 0};
                v[a] = f4{};
                if (i < chunks) {
                    s[a] = stats[uint64_t{i} * per];
                    v[a] = part[uint64_t{i} * per * kQuads];
                }
            }
#pragma unroll
            for (uint32_t a = 0; a < kAhead; ++a) most = fmaxf(most, s[a].x);
            const float from = most == -INFINITY ? 0.0f : most, fade = exp2_(top - from);
            top = most;
            total *= fade;
            o *= fade;
#pragma unroll
            for (uint32_t a = 0; a < kAhead; ++a) {
                const float f = exp2_(s[a].x - from);
                total += s[a].y * f;
                // without positions a chunk's values are not written
                if (s[a].x != -INFINITY || s[a].y != 0) o += v[a] * f;
            }
        }
    }
    if (share > 1) {
        s_part[threadIdx.x] = o;
        s_stat[threadIdx.x] = v2f{top, total};
        __syncthreads();
        if (group) return;
        for (uint32_t g = 1; g < share; ++g) {
            const v2f s = s_stat[threadIdx.x + g * kQuads];
            const float most = fmaxf(top, s.x), from = most == -INFINITY ? 0.0f : most, fade = exp2_(top - from), f = exp2_(s.x - from);
            top = most;
            total = total * fade + s.y * f;
            o = o * fade + s_part[threadIdx.x + g * kQuads] * f;
        }
    }
    if (row >= rows) return;
    if (total == 0) o = f4{};
    const float inv = total == 0 ? 0.0f : 1.0f / total;
    v2u to;
    to.x = pack2b(o[0] * inv, o[1] * inv);
    to.y = pack2b(o[2] * inv, o[3] * inv);
    *reinterpret_cast<v2u *>(p.out + row * kDim + 4 * d) = to;
    if (d == 0 && p.lse) p.lse[row] = ((top == -INFINITY ? 0.0f : top) + __builtin_amdgcn_logf(total)) * kLn2;
}

// ---- Host ------------------------------------------------------------------

// Tiles of 128 rows read K and V half as often as those of 64, but are half as many
// workgroups: they are taken where each still has this many positions.  64 nodes of 32 heads:
// 1 x 32,768 73 us against 80 with 64 rows, 1 x 65,536 E4M3 93 against 98; 8 up to 8,192 with
// 25 nodes 46.9 against 50.2; with fewer positions there are not enough workgroups.
constexpr uint64_t kLargeChunk = 1024;

struct Shape {
    uint32_t rows;  // of a workgroup: 16 and 32 in tree_few_kernel, more in tree_many_kernel
    uint32_t tiles, splits;
    uint64_t chunks;  // of all sequences
    uint32_t share;   // 0: each sequence has as many
};

// Sequences are cut where there are fewer workgroups than run at once (two for each
// compute unit), into chunks of 128 positions at least, a step for each wave.  17 to 32
// rows over heads of 256 take tiles of 64, of which half stay empty: in two tiles of 16,
// which read K and V twice, 1 x 8,192 takes 24.9 us (20.2), 16 x 4,096 71 (66), 8 x 32,768
// E4M3 122 (113), 64 up to 1,000 51 (37), each with 4 cache heads for 8.
Shape shape_of(uint64_t batch, uint64_t nodes, uint32_t group, uint32_t kv_heads, uint32_t dim, uint64_t positions) {
    const uint64_t rows = nodes * group;
    Shape s;
    s.rows = rows <= 16 ? 16 : rows <= 32 && dim < 256 ? 32 : 64;
    const uint64_t large = batch * kv_heads * ((rows + 127) / 128);  // workgroups with all positions
    if (rows > 64 && dim < 256 && large * positions >= 2 * kComputeUnits * kLargeChunk) s.rows = 128;
    s.tiles = static_cast<uint32_t>((rows + s.rows - 1) / s.rows);
    const uint64_t units = batch * kv_heads * s.tiles;
    s.share = 0;
    if (units == 0) {  // no rows: nothing to cut
        s.splits = 1;
        s.chunks = 0;
        return s;
    }
    const uint64_t want = (kSlots + units - 1) / units;
    const uint64_t most = (positions + kMinChunk - 1) / kMinChunk;
    s.splits = static_cast<uint32_t>(positions <= 2 * kMinChunk ? 1 : std::min(want, most));
    s.chunks = batch * s.splits;
    if (s.splits > 1 && batch > 1 && batch <= 64) {  // a lane for each sequence
        const uint64_t at_once = kSlots / (kv_heads * s.tiles);
        s.share = static_cast<uint32_t>(at_once - batch / 2);
        s.chunks = s.share + batch;
    }
    return s;
}

// A cut is made only of sizes that pass: the tiles of fewer than 2^24 rows fit 32 bits.
bool sizes_ok(uint64_t batch, uint64_t nodes, uint32_t q_heads, uint32_t kv_heads, uint32_t page_size, uint64_t width) {
    return batch <= (1u << 24) && nodes <= (1u << 20) && kv_heads > 0 && kv_heads <= 65536 && q_heads > 0 && q_heads <= (1u << 20) &&
           q_heads % kv_heads == 0 && width > 0 && width < (1u << 30) / page_size && span(batch, nodes * q_heads) < (1u << 24);
}

uint64_t workgroups(uint32_t kv_heads, const Shape &s) {
    return (kv_heads * s.chunks + 7) / 8 * 8 * s.tiles;
}

// Whether the kernels' work items fit a launch, which holds fewer than 2^32.
bool launchable(uint32_t kv_heads, const Shape &s) {
    return kv_heads * s.chunks < (uint64_t{1} << 32) && workgroups(kv_heads, s) < (1u << 24);
}

uint64_t workspace_of(uint64_t batch, uint64_t nodes, uint32_t q_heads, uint32_t dim, const Shape &s) {
    return s.splits <= 1 ? 0 : s.chunks * nodes * q_heads * (dim + 2) * sizeof(float) + (s.share ? batch * 2 * sizeof(uint32_t) : 0);
}

template <int kDim>
auto kernel_of(bool e4m3, uint32_t rows) {
    if constexpr (kDim == 256) {
        if (rows == 64) return e4m3 ? tree_many_kernel<kDim, true, 1, 1> : tree_many_kernel<kDim, false, 1, 1>;
    } else {
        if (rows == 32) return e4m3 ? tree_few_kernel<kDim, true, 2> : tree_few_kernel<kDim, false, 2>;
        if (rows == 128) return e4m3 ? tree_many_kernel<kDim, true, 2, 1> : tree_many_kernel<kDim, false, 2, 1>;
        if (rows == 64) return e4m3 ? tree_many_kernel<kDim, true, 2, 2> : tree_many_kernel<kDim, false, 2, 2>;
    }
    return e4m3 ? tree_few_kernel<kDim, true, 1> : tree_few_kernel<kDim, false, 1>;
}

constexpr uint64_t kMaxRow = uint64_t{1} << 28;  // bytes; eight of them are an offset in 32 bits

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
    if (p.k.row >= kMaxRow || p.v.row >= kMaxRow) return DF11_E_INVALID_ARG;
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
    if (!launchable(c->kv_heads, s)) return DF11_E_INVALID_ARG;
    p.tiles = s.tiles;
    p.splits = s.splits;
    p.units = static_cast<uint32_t>(c->kv_heads * s.chunks);
    p.share = s.share;
    if (workspace_bytes < workspace_of(t->batch, t->nodes, t->q_heads, c->head_dim, s)) return DF11_E_BUFFER_TOO_SMALL;
    if (s.splits > 1 && !workspace) return DF11_E_INVALID_ARG;
    const uint64_t rows = t->batch * t->nodes * t->q_heads;
    p.part = static_cast<float *>(workspace);
    const uint64_t parts = s.chunks * t->nodes * t->q_heads;
    p.stats = s.splits > 1 ? p.part + parts * c->head_dim : nullptr;
    p.own = s.share ? reinterpret_cast<uint32_t *>(p.stats + parts * 2) : nullptr;
    const bool e4m3 = c->dtype == DF11_CACHE_E4M3;
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    auto fn = c->head_dim == 64    ? kernel_of<64>(e4m3, s.rows)
              : c->head_dim == 128 ? kernel_of<128>(e4m3, s.rows)
                                   : kernel_of<256>(e4m3, s.rows);
    hipError_t err = launch(fn, static_cast<uint32_t>(workgroups(c->kv_heads, s)), 64 * (s.rows > 32 ? kManyWaves : kWaves), 0, st, p);
    if (err == hipSuccess && s.splits > 1) {
        uint32_t share = 1;
        while (share < kJoinThreads / (c->head_dim / 4) && 4 * share < s.chunks / t->batch) share *= 2;
        const uint64_t per = kJoinThreads / (c->head_dim / 4) / share;
        err = launch(c->head_dim == 64    ? tree_join_kernel<64>
                     : c->head_dim == 128 ? tree_join_kernel<128>
                                          : tree_join_kernel<256>,
                     static_cast<uint32_t>((rows + per - 1) / per), kJoinThreads, 0, st, p, rows, share);
    }
    return launched(err);
}

}  // namespace

extern "C" uint64_t df11_paged_tree_attention_workspace_bytes(uint64_t batch, uint64_t nodes, uint32_t q_heads,
                                                              uint32_t kv_heads, uint32_t head_dim, uint32_t page_size,
                                                              uint64_t table_width) {
    if (!dim_ok(head_dim) || !page_ok(page_size) || !sizes_ok(batch, nodes, q_heads, kv_heads, page_size, table_width)) return 0;
    const Shape s = shape_of(batch, nodes, q_heads / kv_heads, kv_heads, head_dim, table_width * page_size);
    return launchable(kv_heads, s) ? workspace_of(batch, nodes, q_heads, head_dim, s) : 0;
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
