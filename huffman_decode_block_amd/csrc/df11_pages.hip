// Pages of a cache after a choice between candidates (gfx950): copied, made
// contiguous, shared, taken and given back (include/df11_search.h).
#include <hip/hip_runtime.h>

#include <climits>

#include "df11_paged.h"
#include "df11_search.h"

namespace {

using namespace df11p;

// A row's 16-byte pieces, two to the power of this.
uint32_t piece_shift(const df11_paged_cache *c) { return log2_of(c->head_dim * (c->dtype == DF11_CACHE_E4M3 ? 1 : 2) / 16); }

// ---- Copy -------------------------------------------------------------------
// Bytes moved and nothing else: bound by HBM.  A lane has four 16-byte pieces on
// their way, a workgroup 16 KiB of one page's K or V.  2,048 whole E4M3 pages (1.07
// GB read and written): 187 us, 5.8 TB/s; 32 pages in part in 32 layers 11 us.

constexpr uint32_t kThreads = 256;
constexpr int kAhead = 4;  // pieces that a lane has on their way
constexpr uint32_t kPerGroup = kThreads * kAhead;

struct CopyParams {
    Pages k, v;
    uint64_t k_layer, v_layer;  // bytes
    const int32_t *src, *dst, *rows;
    uint64_t n_pages;
    uint32_t n, parts, pieces;  // parts: workgroups for the K (or V) of a page; pieces of it
    uint32_t groups;            // n * layers * 2 * parts
    uint32_t page_shift, piece_shift;
};

__global__ void __launch_bounds__(kThreads) copy_kernel(CopyParams p) {
    for (uint32_t id = blockIdx.x; id < p.groups; id += gridDim.x) {
        const uint32_t pair = id / (2 * p.parts), part = id - pair * 2 * p.parts;
        const uint32_t layer = pair / p.n, i = pair - layer * p.n;
        const bool is_v = part >= p.parts;
        const int32_t from = p.src[i], to = p.dst[i];
        const int32_t rows = p.rows ? p.rows[i] : INT_MAX;
        if (from < 0 || to < 0 || static_cast<uint64_t>(from) >= p.n_pages || static_cast<uint64_t>(to) >= p.n_pages) continue;
        const Pages &x = is_v ? p.v : p.k;
        uint8_t *base = x.base + layer * (is_v ? p.v_layer : p.k_layer);
        const uint8_t *a = base + static_cast<uint64_t>(from) * x.page;
        uint8_t *b = base + static_cast<uint64_t>(to) * x.page;
        const uint32_t at = (is_v ? part - p.parts : part) * kPerGroup + threadIdx.x;
        v4u w[kAhead];
        uint64_t off[kAhead];
        bool have[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint32_t e = at + j * kThreads;
            const uint32_t piece = e & ((1u << p.piece_shift) - 1), row = (e >> p.piece_shift) & ((1u << p.page_shift) - 1);
            const uint32_t head = e >> (p.piece_shift + p.page_shift);
            have[j] = e < p.pieces && static_cast<int32_t>(row) < rows;
            off[j] = head * x.head + row * x.row + 16 * piece;
            if (have[j]) w[j] = *reinterpret_cast<const v4u *>(a + off[j]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (have[j]) *reinterpret_cast<v4u *>(b + off[j]) = w[j];
    }
}

// ---- Compact ----------------------------------------------------------------

constexpr uint32_t kMaxDepth = 1024;
constexpr uint32_t kLanes = 64;

struct CompactParams {
    Pages k, v;
    uint64_t k_layer, v_layer;  // bytes
    const int32_t *path, *accepted, *table, *lens;
    uint64_t table_stride, n_pages;
    uint32_t layers, depth, parts, pieces;  // pieces: 16 bytes of a position's K and V; parts: workgroups for them
    uint32_t groups;                        // batch * layers * parts
    uint32_t page_shift, piece_shift, positions;
};

// A lane moves one piece of all rows, eight at a time: as a path ascends, what
// is written lies in front of what is still to be read.  No barrier is needed
// between rows, as a lane's piece of every row is its own.  One path of a tree of 64
// in 32 layers: 5.1 us, a start and one chain of dependent loads (accepted, path,
// table, rows); 64 paths of E4M3 11.3 us against 8.2 by their bytes.
__global__ void __launch_bounds__(kThreads) compact_kernel(CompactParams p) {
    __shared__ int32_t s_from[kLanes], s_to[kLanes];  // pages; -1: no move
    __shared__ uint32_t s_rows[kLanes];               // rows in them: source, target in the high half
    __shared__ uint32_t s_moves;
    for (uint32_t id = blockIdx.x; id < p.groups; id += gridDim.x) {
        const uint32_t unit = id / p.parts, part = id - unit * p.parts;
        const uint32_t b = unit / p.layers, layer = unit - b * p.layers;
        const uint32_t n = min(static_cast<uint32_t>(max(p.accepted[b], 0)), p.depth);
        const uint32_t len = static_cast<uint32_t>(max(p.lens[b], 0));
        const int32_t *path = p.path + static_cast<uint64_t>(b) * p.depth;
        const int32_t *table = p.table + b * p.table_stride;
        const uint32_t e = part * kThreads + threadIdx.x;
        const bool is_v = e >= p.pieces / 2, have = e < p.pieces;
        const uint32_t in = is_v ? e - p.pieces / 2 : e;
        const uint32_t head = in >> p.piece_shift, piece = in & ((1u << p.piece_shift) - 1);
        const Pages &x = is_v ? p.v : p.k;
        uint8_t *base = x.base + layer * (is_v ? p.v_layer : p.k_layer) + head * x.head + 16 * piece;
        for (uint32_t i0 = 0; i0 < n; i0 += kLanes) {
            if (threadIdx.x < kLanes) {
                const uint32_t i = i0 + threadIdx.x;
                const int32_t at = i < n ? path[i] : -1, before = i > 0 && i < n ? path[i - 1] : -1;
                const uint64_t ends = __ballot(at < 0 || at <= before);
                const uint32_t moves = ends ? __builtin_ctzll(ends) : kLanes;
                const uint64_t from = uint64_t{len} + static_cast<uint32_t>(max(at, 0)), to = uint64_t{len} + i;
                int32_t page = -1, to_page = -1;
                if (threadIdx.x < moves && from != to && from < p.positions) {
                    page = table[from >> p.page_shift];
                    to_page = table[to >> p.page_shift];
                }
                const bool ok = page >= 0 && to_page >= 0 && static_cast<uint64_t>(page) < p.n_pages &&
                                static_cast<uint64_t>(to_page) < p.n_pages;
                const uint32_t mask = (1u << p.page_shift) - 1;
                s_from[threadIdx.x] = ok ? page : -1;
                s_to[threadIdx.x] = ok ? to_page : -1;
                s_rows[threadIdx.x] = (static_cast<uint32_t>(from) & mask) | (static_cast<uint32_t>(to) & mask) << 16;
                if (threadIdx.x == 0) s_moves = moves;
            }
            __syncthreads();
            const uint32_t moves = s_moves;
            if (have)
                for (uint32_t j0 = 0; j0 < moves; j0 += 8) {
                    v4u w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j0 + j < moves && s_from[j0 + j] >= 0)
                            w[j] = *reinterpret_cast<const v4u *>(base + static_cast<uint64_t>(s_from[j0 + j]) * x.page +
                                                                  uint64_t{s_rows[j0 + j] & 0xFFFFu} * x.row);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j0 + j < moves && s_from[j0 + j] >= 0)
                            *reinterpret_cast<v4u *>(base + static_cast<uint64_t>(s_to[j0 + j]) * x.page +
                                                     uint64_t{s_rows[j0 + j] >> 16} * x.row) = w[j];
                }
            __syncthreads();
            if (moves < kLanes) break;
        }
    }
}

// ---- Fork -------------------------------------------------------------------
// Two kernels.  One workgroup plans: it finds for every row the pages that it
// has to have for itself, keeps its parent's where it may, and gives it free
// ones.  Then workgroups of four columns each move the entries through LDS and
// count: one that changes takes a holder from the old page and gives one to the
// new.  Counts are whole numbers, so that the order of the atomics does not matter.
// One workgroup for the plan, as a row's pages depend on what the rows before it
// took; it looks at 16 pages of the pool in each lane at a time, and at four entries.
// Bound by latency, chains of parent, table, count: 6.9 + 3.7 us for 32 rows, 12.2 +
// 7.4 for 512 rows of up to 8,100 positions over 513 columns (an entry at a time for
// each lane: 6.4 + 3.3 and 13.8 + 10.5).

constexpr uint32_t kMaxBatch = 4096;
constexpr uint32_t kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;
constexpr int kPlanAhead = 16;  // pages that a lane looks at together
constexpr uint32_t kColumns = 4;
constexpr uint32_t kRowsAhead = 4;   // entries that a lane of the plan looks at together
constexpr uint32_t kTableAhead = 2;  // rows that one of the table does

struct ForkParams {
    const int32_t *parents;
    int32_t *table, *lens, *refs, *src, *dst, *rows, *missing;
    int32_t *own;    // [batch][columns]: pages from column L / page_size on
    int32_t *fresh;  // [batch * columns]: free pages
    uint64_t table_stride, n_pages;
    uint32_t batch, width, columns, room, page_shift;
};

__device__ __forceinline__ int32_t parent_of(const ForkParams &p, uint32_t b) {
    const int32_t a = p.parents ? p.parents[b] : static_cast<int32_t>(b);
    return a >= 0 && static_cast<uint32_t>(a) < p.batch ? a : -1;
}

__device__ __forceinline__ bool is_page(const ForkParams &p, int32_t e) { return e >= 0 && static_cast<uint64_t>(e) < p.n_pages; }

// Columns that a row of L positions has to have.
__device__ __forceinline__ uint32_t columns_of(const ForkParams &p, uint32_t len) {
    return min((len + p.room + (1u << p.page_shift) - 1) >> p.page_shift, p.width);
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(ForkParams p) {
    __shared__ int32_t s_first[kMaxBatch];  // the lowest row that goes on from a row
    __shared__ uint32_t s_len[kMaxBatch];
    __shared__ uint32_t s_count[kPlanAhead * kPlanWaves + 1];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const auto before = [&](uint64_t mask) {
        return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
    };
    for (uint32_t b = threadIdx.x; b < p.batch; b += kPlanThreads) {
        s_first[b] = INT_MAX;
        s_len[b] = min(static_cast<uint32_t>(max(p.lens[b], 0)), p.width << p.page_shift);
    }
    __syncthreads();
    for (uint32_t b = threadIdx.x; b < p.batch; b += kPlanThreads) {
        const int32_t a = parent_of(p, b);
        if (a >= 0) atomicMin(&s_first[a], static_cast<int32_t>(b));
    }
    __syncthreads();

    // own pages, in order: kept ones, and -2 - n for the n-th that is wanted
    uint32_t wants = 0;
    const uint32_t entries = p.batch * p.columns;
    for (uint32_t e0 = 0; e0 < entries; e0 += kRowsAhead * kPlanThreads) {
        int32_t a[kRowsAhead], page[kRowsAhead], holders[kRowsAhead];
        uint32_t want = 0, keep = 0;  // a bit for each
        uint64_t mask[kRowsAhead];
#pragma unroll
        for (uint32_t h = 0; h < kRowsAhead; ++h) {
            a[h] = -1;
            if (e0 + h * kPlanThreads < entries) a[h] = parent_of(p, min(e0 + h * kPlanThreads + threadIdx.x, entries - 1) / p.columns);
        }
#pragma unroll
        for (uint32_t h = 0; h < kRowsAhead; ++h) {
            const uint32_t e = e0 + h * kPlanThreads + threadIdx.x, b = e / p.columns;
            page[h] = -1;
            if (e0 + h * kPlanThreads >= entries) continue;
            if (e < entries && a[h] >= 0) {
                const uint32_t len = s_len[a[h]], col = (len >> p.page_shift) + (e - b * p.columns);
                if (col < columns_of(p, len)) {
                    want |= 1u << h;
                    if (s_first[a[h]] == static_cast<int32_t>(b)) page[h] = p.table[a[h] * p.table_stride + col];
                }
            }
        }
#pragma unroll
        for (uint32_t h = 0; h < kRowsAhead; ++h) {
            holders[h] = 2;
            if (e0 + h * kPlanThreads < entries && is_page(p, page[h])) holders[h] = p.refs[page[h]];
        }
#pragma unroll
        for (uint32_t h = 0; h < kRowsAhead; ++h) {
            keep |= (holders[h] <= 1) << h;
            want &= ~keep;
            mask[h] = __ballot(want >> h & 1u);
            if (lane == 0) s_count[h * kPlanWaves + wave] = __popcll(mask[h]);
        }
        __syncthreads();
        // what comes before each of the 64 counts, a lane's each
        static_assert(kRowsAhead * kPlanWaves == 64, "a lane for each count");
        const uint32_t mine = s_count[lane], upto = df11w::wave_inclusive_scan(mine);
#pragma unroll
        for (uint32_t h = 0; h < kRowsAhead; ++h) {
            const uint32_t e = e0 + h * kPlanThreads + threadIdx.x;
            const uint32_t at = wants + __builtin_amdgcn_readlane(upto - mine, h * kPlanWaves + wave) + before(mask[h]);
            if (e < entries) p.own[e] = want >> h & 1u ? -2 - static_cast<int32_t>(at) : keep >> h & 1u ? page[h] : -1;
        }
        wants += __builtin_amdgcn_readlane(upto, 63);
        __syncthreads();
    }

    // free pages in their order, as many as are wanted
    uint32_t found = 0;
    for (uint64_t base = 0; base < p.n_pages && found < wants; base += kPlanAhead * kPlanThreads) {
        uint32_t is_free = 0;
        uint64_t mask[kPlanAhead];
#pragma unroll
        for (int j = 0; j < kPlanAhead; ++j) {
            const uint64_t page = base + j * kPlanThreads + threadIdx.x;
            const bool yes = page < p.n_pages && p.refs[page] == 0;
            is_free |= static_cast<uint32_t>(yes) << j;
        }
#pragma unroll
        for (int j = 0; j < kPlanAhead; ++j) {
            mask[j] = __ballot(is_free >> j & 1u);
            if (lane == 0) s_count[j * kPlanWaves + wave] = __popcll(mask[j]);
        }
        __syncthreads();
        // what comes before each of the counts
        constexpr uint32_t kCounts = kPlanAhead * kPlanWaves;
        if (wave == 0) {
            uint32_t n[kCounts / 64], sum = 0;
#pragma unroll
            for (uint32_t j = 0; j < kCounts / 64; ++j) {
                n[j] = s_count[lane * (kCounts / 64) + j];
                sum += n[j];
            }
            uint32_t at = df11w::wave_inclusive_scan(sum);
            if (lane == 63) s_count[kCounts] = at;
            at -= sum;
#pragma unroll
            for (uint32_t j = 0; j < kCounts / 64; ++j) {
                s_count[lane * (kCounts / 64) + j] = at;
                at += n[j];
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPlanAhead; ++j) {
            const uint32_t at = found + s_count[j * kPlanWaves + wave] + before(mask[j]);
            if ((is_free >> j & 1u) && at < wants) p.fresh[at] = static_cast<int32_t>(base + j * kPlanThreads + threadIdx.x);
        }
        found += s_count[kCounts];
        __syncthreads();
    }
    found = min(found, wants);
    __syncthreads();

    for (uint32_t e0 = threadIdx.x; e0 < entries; e0 += kRowsAhead * kPlanThreads) {
        int32_t own[kRowsAhead], page[kRowsAhead];
#pragma unroll
        for (uint32_t h = 0; h < kRowsAhead; ++h) {
            own[h] = -1;
            if (e0 + h * kPlanThreads < entries) own[h] = p.own[e0 + h * kPlanThreads];
        }
#pragma unroll
        for (uint32_t h = 0; h < kRowsAhead; ++h) {
            const uint32_t n = static_cast<uint32_t>(-2 - own[h]);
            page[h] = own[h] <= -2 && n < found ? p.fresh[n] : -1;
        }
#pragma unroll
        for (uint32_t h = 0; h < kRowsAhead; ++h)
            if (e0 + h * kPlanThreads < entries && own[h] <= -2) p.own[e0 + h * kPlanThreads] = page[h];
    }
    __syncthreads();
    for (uint32_t b = threadIdx.x; b < p.batch; b += kPlanThreads) {
        const int32_t a = parent_of(p, b);
        int32_t src = -1, dst = -1, rows = 0;
        uint32_t len = 0;
        if (a >= 0) {
            len = s_len[a];
            const uint32_t filled = len & ((1u << p.page_shift) - 1);
            if (filled) {
                const int32_t old = p.table[a * p.table_stride + (len >> p.page_shift)], now = p.own[uint64_t{b} * p.columns];
                if (is_page(p, old) && now >= 0 && now != old) {
                    src = old;
                    dst = now;
                    rows = static_cast<int32_t>(filled);
                }
            }
        }
        p.src[b] = src;
        p.dst[b] = dst;
        p.rows[b] = rows;
        p.lens[b] = static_cast<int32_t>(len);
    }
    if (threadIdx.x == 0) p.missing[0] = static_cast<int32_t>(wants - found);
}

__global__ void __launch_bounds__(kThreads) fork_table_kernel(ForkParams p) {
    extern __shared__ int32_t s_table[];  // [batch][kColumns]
    const uint32_t col0 = blockIdx.x * kColumns;
    const uint32_t there = min(kColumns, p.width - col0);
    // a thread's rows, all their columns at a time: loads of two rows are on their way together
    for (uint32_t b0 = threadIdx.x; b0 < p.batch; b0 += kTableAhead * kThreads) {
        int32_t e[kTableAhead][kColumns];
#pragma unroll
        for (uint32_t h = 0; h < kTableAhead; ++h) {
            if (h * kThreads >= p.batch) break;
#pragma unroll
            for (uint32_t c = 0; c < kColumns; ++c)
                e[h][c] = p.table[min(b0 + h * kThreads, p.batch - 1) * p.table_stride + col0 + min(c, there - 1)];
        }
#pragma unroll
        for (uint32_t h = 0; h < kTableAhead; ++h)
#pragma unroll
            for (uint32_t c = 0; c < kColumns; ++c)
                if (b0 + h * kThreads < p.batch) s_table[(b0 + h * kThreads) * kColumns + c] = e[h][c];
    }
    __syncthreads();
    for (uint32_t b0 = threadIdx.x; b0 < p.batch; b0 += kTableAhead * kThreads) {
        int32_t a[kTableAhead], own[kTableAhead][kColumns];
        uint32_t len[kTableAhead];
#pragma unroll
        for (uint32_t h = 0; h < kTableAhead; ++h) {
            a[h] = -1;
            len[h] = 0;
            if (h * kThreads >= p.batch) continue;
            const uint32_t b = min(b0 + h * kThreads, p.batch - 1);
            a[h] = parent_of(p, b);
            len[h] = static_cast<uint32_t>(p.lens[b]);
        }
#pragma unroll
        for (uint32_t h = 0; h < kTableAhead; ++h) {
            const uint32_t b = min(b0 + h * kThreads, p.batch - 1), full = len[h] >> p.page_shift, ends = columns_of(p, len[h]);
#pragma unroll
            for (uint32_t c = 0; c < kColumns; ++c) {
                const uint32_t col = col0 + c;
                own[h][c] = -1;
                if (a[h] >= 0 && col >= full && col < ends) own[h][c] = p.own[uint64_t{b} * p.columns + (col - full)];
            }
        }
#pragma unroll
        for (uint32_t h = 0; h < kTableAhead; ++h) {
            const uint32_t b = b0 + h * kThreads, full = len[h] >> p.page_shift;
            if (b >= p.batch) break;
#pragma unroll
            for (uint32_t c = 0; c < kColumns; ++c) {
                if (c >= there) break;
                const int32_t old = s_table[b * kColumns + c];
                int32_t now = own[h][c];
                if (a[h] >= 0 && col0 + c < full) {
                    now = s_table[static_cast<uint32_t>(a[h]) * kColumns + c];
                    if (!is_page(p, now)) now = -1;
                }
                if (now == old) continue;
                p.table[b * p.table_stride + col0 + c] = now;
                if (now >= 0) atomicAdd(&p.refs[now], 1);
                if (is_page(p, old)) atomicSub(&p.refs[old], 1);
            }
        }
    }
}

// ---- Host -------------------------------------------------------------------

// Layers that begin at these strides: multiples of 16 bytes within the limit of addresses.
bool layers_ok(const df11_paged_cache *c, uint32_t layers, uint64_t k_layer, uint64_t v_layer) {
    const uint64_t unit = c->dtype == DF11_CACHE_E4M3 ? 16 : 8;
    if (layers == 0 || layers > 65535 || k_layer % unit || v_layer % unit || k_layer > kMaxStride || v_layer > kMaxStride) return false;
    const auto fits = [&](uint64_t layer, uint64_t page, uint64_t head, uint64_t row) {
        return span(layers, layer) + span(c->n_pages, page) + span(c->kv_heads, head) + span(c->page_size, row) < kMaxExtent;
    };
    return fits(k_layer, c->k_page_stride, c->k_head_stride, c->k_row_stride) &&
           fits(v_layer, c->v_page_stride, c->v_head_stride, c->v_row_stride);
}

// check_cache for calls that look at no scales.
df11_status check_pages(const df11_paged_cache *c) {
    if (!c) return DF11_E_INVALID_ARG;
    df11_paged_cache scaled = *c;
    static const float one = 1;
    scaled.k_scale = scaled.v_scale = &one;
    return check_cache(&scaled);
}

constexpr uint64_t kMostGroups = uint64_t{1} << 20;  // of a launch; kernels go on from there

df11_status copy(const df11_paged_cache *c, uint32_t layers, uint64_t k_layer, uint64_t v_layer, const int32_t *src,
                 const int32_t *dst, const int32_t *rows, uint64_t n, void *hip_stream) {
    const df11_status rc = check_pages(c);
    if (rc != DF11_OK) return rc;
    if (!layers_ok(c, layers, k_layer, v_layer) || n > 0x7FFFFFFFu) return DF11_E_INVALID_ARG;
    if (n == 0) return DF11_OK;
    if (!src || !dst || ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(rows)) & 3u))
        return DF11_E_INVALID_ARG;
    CopyParams p;
    p.k = k_of(c);
    p.v = v_of(c);
    const uint64_t size = c->dtype == DF11_CACHE_E4M3 ? 1 : 2;
    p.k_layer = k_layer * size;
    p.v_layer = v_layer * size;
    p.src = src;
    p.dst = dst;
    p.rows = rows;
    p.n_pages = c->n_pages;
    p.n = static_cast<uint32_t>(n);
    p.page_shift = log2_of(c->page_size);
    p.piece_shift = piece_shift(c);
    p.pieces = c->kv_heads << (p.page_shift + p.piece_shift);  // at most 2^16 * 2^10 * 2^5
    p.parts = (p.pieces + kPerGroup - 1) / kPerGroup;
    const uint64_t pairs = n * layers;
    if (pairs > 0x7FFFFFFFu / (2 * p.parts)) return DF11_E_INVALID_ARG;
    p.groups = static_cast<uint32_t>(pairs * 2 * p.parts);
    return launched(launch(copy_kernel, static_cast<uint32_t>(std::min<uint64_t>(p.groups, kMostGroups)), kThreads, 0,
                           static_cast<hipStream_t>(hip_stream), p));
}

df11_status compact(const df11_paged_cache *c, uint32_t layers, uint64_t k_layer, uint64_t v_layer, const int32_t *path,
                    uint32_t depth, const int32_t *accepted, const int32_t *table, uint64_t table_stride, uint64_t width,
                    const int32_t *lens, uint64_t batch, void *hip_stream) {
    const df11_status rc = check_pages(c);
    if (rc != DF11_OK) return rc;
    if (!layers_ok(c, layers, k_layer, v_layer) || depth > kMaxDepth || width == 0 || width > 0x7FFFFFFFu / c->page_size ||
        table_stride < width || table_stride > kMaxStride || batch > 0x7FFFFFFFu || span(batch, table_stride) >= kMaxExtent)
        return DF11_E_INVALID_ARG;
    if (batch == 0 || depth == 0) return DF11_OK;
    const auto low = [](const void *x) { return reinterpret_cast<uintptr_t>(x); };
    if (!path || !accepted || !table || !lens || ((low(path) | low(accepted) | low(table) | low(lens)) & 3u)) return DF11_E_INVALID_ARG;
    CompactParams p;
    p.k = k_of(c);
    p.v = v_of(c);
    const uint64_t size = c->dtype == DF11_CACHE_E4M3 ? 1 : 2;
    p.k_layer = k_layer * size;
    p.v_layer = v_layer * size;
    p.path = path;
    p.accepted = accepted;
    p.table = table;
    p.lens = lens;
    p.table_stride = table_stride;
    p.n_pages = c->n_pages;
    p.layers = layers;
    p.depth = depth;
    p.page_shift = log2_of(c->page_size);
    p.piece_shift = piece_shift(c);
    p.positions = static_cast<uint32_t>(width * c->page_size);
    p.pieces = 2 * c->kv_heads << p.piece_shift;
    p.parts = (p.pieces + kThreads - 1) / kThreads;
    const uint64_t units = batch * layers;
    if (units > 0x7FFFFFFFu / p.parts) return DF11_E_INVALID_ARG;
    p.groups = static_cast<uint32_t>(units * p.parts);
    return launched(launch(compact_kernel, static_cast<uint32_t>(std::min<uint64_t>(p.groups, kMostGroups)), kThreads, 0,
                           static_cast<hipStream_t>(hip_stream), p));
}

// Columns from L / page_size on that a row may own.
uint64_t own_columns(uint64_t width, uint32_t page_size, uint64_t room) {
    return std::min<uint64_t>((room + 2 * uint64_t{page_size} - 2) / page_size, width);
}

bool fork_sizes_ok(uint64_t batch, uint64_t width, uint32_t page_size, uint64_t n_pages, uint64_t room) {
    return batch <= kMaxBatch && page_ok(page_size) && width > 0 && width <= (1u << 24) && width <= 0x7FFFFFFFu / page_size &&
           n_pages > 0 && n_pages <= 0x7FFFFFFFu && room <= (1u << 30) &&
           batch * own_columns(width, page_size, room) <= (1u << 30);
}

df11_status fork(const int32_t *parents, uint64_t batch, int32_t *table, uint64_t table_stride, uint64_t width,
                 uint32_t page_size, int32_t *lens, int32_t *refs, uint64_t n_pages, uint64_t room, int32_t *src,
                 int32_t *dst, int32_t *rows, int32_t *missing, void *workspace, uint64_t workspace_bytes,
                 void *hip_stream) {
    if (!fork_sizes_ok(batch, width, page_size, n_pages, room) || table_stride < width || table_stride > (uint64_t{1} << 32))
        return DF11_E_INVALID_ARG;
    const auto low = [](const void *x) { return reinterpret_cast<uintptr_t>(x); };
    if (!missing || ((low(parents) | low(table) | low(lens) | low(refs) | low(src) | low(dst) | low(rows) | low(missing)) & 3u) ||
        !aligned16(workspace))
        return DF11_E_INVALID_ARG;
    if (batch && (!table || !lens || !refs || !src || !dst || !rows)) return DF11_E_INVALID_ARG;
    const uint64_t columns = own_columns(width, page_size, room);
    if (workspace_bytes < df11_paged_fork_workspace_bytes(batch, width, page_size, n_pages, room)) return DF11_E_BUFFER_TOO_SMALL;
    if (batch && !workspace) return DF11_E_INVALID_ARG;
    ForkParams p;
    p.parents = parents;
    p.table = table;
    p.lens = lens;
    p.refs = refs;
    p.src = src;
    p.dst = dst;
    p.rows = rows;
    p.missing = missing;
    p.own = static_cast<int32_t *>(workspace);
    p.fresh = p.own + batch * columns;
    p.table_stride = table_stride;
    p.n_pages = n_pages;
    p.batch = static_cast<uint32_t>(batch);
    p.width = static_cast<uint32_t>(width);
    p.columns = static_cast<uint32_t>(columns);
    p.room = static_cast<uint32_t>(room);
    p.page_shift = log2_of(page_size);
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    hipError_t err = launch(fork_plan_kernel, 1, kPlanThreads, 0, st, p);
    if (err == hipSuccess && batch)
        err = launch(fork_table_kernel, static_cast<uint32_t>((width + kColumns - 1) / kColumns), kThreads,
                     static_cast<uint32_t>(batch * kColumns * sizeof(int32_t)), st, p);
    return launched(err);
}

}  // namespace

extern "C" df11_status df11_paged_copy(const df11_paged_cache *cache, uint32_t layers, uint64_t k_layer_stride,
                                       uint64_t v_layer_stride, const int32_t *src, const int32_t *dst,
                                       const int32_t *rows, uint64_t n, void *hip_stream) {
    return df11i::guarded([&] { return copy(cache, layers, k_layer_stride, v_layer_stride, src, dst, rows, n, hip_stream); });
}

extern "C" df11_status df11_paged_compact(const df11_paged_cache *cache, uint32_t layers, uint64_t k_layer_stride,
                                          uint64_t v_layer_stride, const int32_t *path, uint32_t depth,
                                          const int32_t *accepted, const int32_t *page_table, uint64_t table_stride,
                                          uint64_t table_width, const int32_t *lens, uint64_t batch, void *hip_stream) {
    return df11i::guarded([&] {
        return compact(cache, layers, k_layer_stride, v_layer_stride, path, depth, accepted, page_table, table_stride,
                       table_width, lens, batch, hip_stream);
    });
}

extern "C" uint64_t df11_paged_fork_workspace_bytes(uint64_t batch, uint64_t table_width, uint32_t page_size,
                                                    uint64_t n_pages, uint64_t room) {
    if (!fork_sizes_ok(batch, table_width, page_size, n_pages, room)) return 0;
    return batch * own_columns(table_width, page_size, room) * 2 * sizeof(int32_t);
}

extern "C" df11_status df11_paged_fork(const int32_t *parents, uint64_t batch, int32_t *page_table,
                                       uint64_t table_stride, uint64_t table_width, uint32_t page_size, int32_t *lens,
                                       int32_t *refs, uint64_t n_pages, uint64_t room, int32_t *src, int32_t *dst,
                                       int32_t *rows, int32_t *missing, void *workspace, uint64_t workspace_bytes,
                                       void *hip_stream) {
    return df11i::guarded([&] {
        return fork(parents, batch, page_table, table_stride, table_width, page_size, lens, refs, n_pages, room, src, dst, rows,
                    missing, workspace, workspace_bytes, hip_stream);
    });
}
