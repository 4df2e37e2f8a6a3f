// Selection of a beam search (gfx950): the best continuations of each search's
// beams over a vocabulary (include/df11_search.h).
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>

#include "df11_paged.h"
#include "df11_search.h"

namespace {

using namespace df11p;

// Two kernels.  In the first a workgroup takes a part of a beam's logits into
// registers, whole: their maximum, their sum of exponentials, and the k best.
// The second adds the parts' sums to each beam's logarithm and chooses among
// all parts' best ones.
//
// Choosing k of n: with t the k-th largest of 64 lanes' largest values, at least
// k values reach t, and few more do; they go to LDS in any order, and each counts
// those before it.  t is sought bit by bit, half of the bits (a value that is
// lower than the k-th largest only lets more values through).

constexpr uint32_t kThreads = 256, kWaves = kThreads / 64;
constexpr uint32_t kMaxK = 64;
constexpr uint32_t kRoom = 1024;  // values that may reach t before they are sought one by one
constexpr uint32_t kEach = 8;     // values of a load

struct BeamParams {
    const void *logits;
    const float *scores;
    const uint8_t *done;
    float *out_scores;
    int32_t *out_parents, *out_tokens;
    float *best;    // [rows][parts][k]: logits, best first; -infinity where there are fewer
    int32_t *at;    // [rows][parts][k]: their tokens
    float *sums;    // [rows][parts][2]: maximum, sum of exp(x - maximum)
    uint64_t batch_stride, beam_stride;
    uint32_t beams, vocab, k, parts, part;  // part: tokens in each
    int32_t pad;
};

// A whole number in the order of the floats, NaN aside.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float of_key(uint32_t k) { return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// A value that at least k lanes' reach (-infinity where fewer have more), near the k-th largest.
__device__ __forceinline__ float reached_by(float x, uint32_t k) {
    const uint32_t key = key_of(x);
    uint32_t t = 0;
#pragma unroll
    for (int bit = 31; bit >= 16; --bit) {
        const uint32_t with = t | 1u << bit;
        if (__popcll(__ballot(key >= with)) >= k) t = with;
    }
    return fmaxf(of_key(t), -INFINITY);  // NaN for keys below that of -infinity
}

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

struct __attribute__((packed, aligned(4))) EightFloats {
    float x[8];
};

// Eight tokens' logits from `at` on; -infinity from `end` on.
template <bool kF32>
__device__ __forceinline__ void load_logits(const void *row, uint32_t at, uint32_t end, float (&x)[kEach]) {
    if (at + kEach <= end) {
        if (kF32) {
            const EightFloats w = *reinterpret_cast<const EightFloats *>(static_cast<const float *>(row) + at);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = w.x[i];
        } else {
            const v4u w = load8(static_cast<const uint16_t *>(row) + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __builtin_bit_cast(float, w[i] << 16);
                x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = -INFINITY;
            if (at + i < end)
                x[i] = kF32 ? static_cast<const float *>(row)[at + i]
                            : __builtin_bit_cast(float, uint32_t{static_cast<const uint16_t *>(row)[at + i]} << 16);
        }
    }
}

template <bool kF32, int kLoads>
__global__ void __launch_bounds__(kThreads) beam_part_kernel(BeamParams p) {
    __shared__ float s_max[kWaves], s_sum[kWaves], s_reach[kWaves];
    __shared__ float s_x[kRoom];
    __shared__ uint32_t s_at[kRoom];
    __shared__ uint32_t s_n;
    const uint32_t row = blockIdx.x / p.parts, part = blockIdx.x - row * p.parts;
    if (p.done && p.done[row]) return;
    if (!(fabsf(p.scores[row]) < INFINITY)) return;
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t b = row / p.beams;
    const uint64_t first = b * p.batch_stride + (row - b * p.beams) * p.beam_stride;
    const void *logits = static_cast<const uint8_t *>(p.logits) + first * (kF32 ? 4 : 2);
    const uint32_t begin = part * p.part, end = min(begin + p.part, p.vocab);

    float x[kLoads][kEach];
    const auto token = [&](int i, int j) { return begin + (i * kThreads + threadIdx.x) * kEach + j; };
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load_logits<kF32>(logits, token(i, 0), end, x[i]);
    float top = -INFINITY;  // NaN aside, which makes the sum NaN
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int j = 0; j < static_cast<int>(kEach); ++j) top = fmaxf(top, x[i][j]);
    const float reach = reached_by(top, p.k), wave_top = wave_max(top);
    if (lane == 0) {
        s_max[wave] = wave_top;
        s_reach[wave] = reach;
    }
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    float m = s_max[0], t = s_reach[0];
#pragma unroll
    for (uint32_t w = 1; w < kWaves; ++w) {
        m = fmaxf(m, s_max[w]);
        t = fmaxf(t, s_reach[w]);
    }
    const float from = m == -INFINITY ? 0.0f : m;
    float sum = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        float e[kEach];
#pragma unroll
        for (int j = 0; j < static_cast<int>(kEach); ++j) e[j] = exp2_((x[i][j] - from) * kLog2e);
        sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    }
    sum = wave_sum(sum);
    if (lane == 0) s_sum[wave] = sum;

    // values that reach t
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int j = 0; j < static_cast<int>(kEach); ++j)
            if (x[i][j] >= t && x[i][j] > -INFINITY) {
                const uint32_t n = atomicAdd(&s_n, 1u);
                if (n < kRoom) {
                    s_x[n] = x[i][j];
                    s_at[n] = token(i, j);
                }
            }
    __syncthreads();
    uint32_t n = s_n;
    const uint64_t out = (uint64_t{row} * p.parts + part) * p.k;
    if (threadIdx.x == 0) {
        float total = 0;
#pragma unroll
        for (uint32_t w = 0; w < kWaves; ++w) total += s_sum[w];
        p.sums[2 * (uint64_t{row} * p.parts + part)] = m;
        p.sums[2 * (uint64_t{row} * p.parts + part) + 1] = total;
    }
    if (n > kRoom) {
        // too many that are equal, or nearly so: the best one k times, each behind the last
        __shared__ float s_best[kWaves];
        __shared__ uint32_t s_best_at[kWaves];
        float last = INFINITY;
        uint32_t last_at = 0;
        bool started = false;
        for (uint32_t i_out = 0; i_out < p.k; ++i_out) {
            float best = -INFINITY;
            uint32_t best_at = UINT_MAX;
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
#pragma unroll
                for (int j = 0; j < static_cast<int>(kEach); ++j) {
                    const uint32_t at = token(i, j);
                    const bool left = x[i][j] > -INFINITY && (!started || x[i][j] < last || (x[i][j] == last && at > last_at));
                    if (left && x[i][j] > best) {
                        best = x[i][j];
                        best_at = at;
                    }
                }
            for (int i = 32; i; i >>= 1) {
                const float o = __shfl_xor(best, i);
                const uint32_t o_at = __shfl_xor(best_at, i);
                if (o > best || (o == best && o_at < best_at)) {
                    best = o;
                    best_at = o_at;
                }
            }
            if (lane == 0) {
                s_best[wave] = best;
                s_best_at[wave] = best_at;
            }
            __syncthreads();
            for (uint32_t w = 0; w < kWaves; ++w)
                if (s_best[w] > best || (s_best[w] == best && s_best_at[w] < best_at)) {
                    best = s_best[w];
                    best_at = s_best_at[w];
                }
            if (threadIdx.x == 0) {
                p.best[out + i_out] = best;
                p.at[out + i_out] = static_cast<int32_t>(best_at);
            }
            last = best;
            last_at = best_at;
            started = true;
            __syncthreads();
        }
        return;
    }
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
        const float v = s_x[i];
        const uint32_t at = s_at[i];
        uint32_t rank = 0;
        for (uint32_t j = 0; j < n; ++j) rank += s_x[j] > v || (s_x[j] == v && s_at[j] < at);
        if (rank < p.k) {
            p.best[out + rank] = v;
            p.at[out + rank] = static_cast<int32_t>(at);
        }
    }
    for (uint32_t i = n + threadIdx.x; i < p.k; i += kThreads) p.best[out + i] = -INFINITY;
}

// A candidate: the score, and what decides between equal ones.
struct Candidate {
    double score;
    uint32_t beam;
    float x;
    uint32_t token;
};

__device__ __forceinline__ bool better(const Candidate &a, const Candidate &b) {
    if (a.score != b.score) return a.score > b.score;
    if (a.beam != b.beam) return a.beam < b.beam;
    if (a.x != b.x) return a.x > b.x;
    return a.token < b.token;
}

constexpr uint32_t kMaxBeams = 1024;

__global__ void __launch_bounds__(kThreads) beam_choose_kernel(BeamParams p) {
    __shared__ double s_lse[kMaxBeams];  // NaN for a beam that offers no token
    __shared__ double s_score[kRoom];
    __shared__ float s_x[kRoom];
    __shared__ uint32_t s_beam[kRoom], s_token[kRoom];
    __shared__ float s_reach[kWaves];
    __shared__ uint32_t s_n;
    const uint32_t b = blockIdx.x, lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint64_t row0 = uint64_t{b} * p.beams;

    for (uint32_t i = wave; i < p.beams; i += kWaves) {
        const uint64_t row = row0 + i;
        const bool open = !(p.done && p.done[row]) && fabsf(p.scores[row]) < INFINITY;
        double lse = NAN;
        if (open) {
            const v2f *sums = reinterpret_cast<const v2f *>(p.sums) + row * p.parts;
            float m = -INFINITY;
            for (uint32_t c = lane; c < p.parts; c += 64) m = fmaxf(m, sums[c].x);
            m = wave_max(m);
            double sum = 0;
            for (uint32_t c = lane; c < p.parts; c += 64) {
                const v2f s = sums[c];
                sum += s.x == -INFINITY ? static_cast<double>(s.y != s.y ? NAN : 0.0f)
                                        : static_cast<double>(s.y) * exp(static_cast<double>(s.x) - static_cast<double>(m));
            }
            for (int k = 32; k; k >>= 1) sum += __shfl_xor(sum, k);
            lse = static_cast<double>(m) + log(sum);
        }
        if (lane == 0) s_lse[i] = lse;
    }
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();

    // candidate c: place c % k of part c / k of a beam; a beam that has ended has one, its first
    const uint32_t per_beam = p.parts * p.k, all = per_beam * p.beams;
    const auto candidate = [&](uint32_t c, Candidate &out) {
        const uint32_t beam = c / per_beam;
        const uint64_t row = row0 + beam;
        out.beam = beam;
        if (p.done && p.done[row]) {
            out.score = p.scores[row];
            out.x = 0;
            out.token = static_cast<uint32_t>(p.pad);
            return c == beam * per_beam && fabsf(p.scores[row]) < INFINITY;
        }
        const double lse = s_lse[beam];
        if (!(fabs(lse) < INFINITY)) return false;
        const uint64_t at = row * per_beam + (c - beam * per_beam);
        out.x = p.best[at];
        if (!(out.x > -INFINITY)) return false;
        out.token = static_cast<uint32_t>(p.at[at]);
        out.score = static_cast<double>(p.scores[row]) + (static_cast<double>(out.x) - lse);
        return true;
    };
    float top = -INFINITY;
    for (uint32_t c = threadIdx.x; c < all; c += kThreads) {
        Candidate x;
        if (candidate(c, x)) top = fmaxf(top, static_cast<float>(x.score));
    }
    const float reach = reached_by(top, p.k);
    if (lane == 0) s_reach[wave] = reach;
    __syncthreads();
    float t = s_reach[0];
#pragma unroll
    for (uint32_t w = 1; w < kWaves; ++w) t = fmaxf(t, s_reach[w]);
    for (uint32_t c = threadIdx.x; c < all; c += kThreads) {
        Candidate x;
        if (candidate(c, x) && static_cast<float>(x.score) >= t) {
            const uint32_t n = atomicAdd(&s_n, 1u);
            if (n < kRoom) {
                s_score[n] = x.score;
                s_beam[n] = x.beam;
                s_x[n] = x.x;
                s_token[n] = x.token;
            }
        }
    }
    __syncthreads();
    const uint32_t n = s_n;
    const uint64_t out = uint64_t{b} * p.k;
    const auto write = [&](uint32_t i, const Candidate &x) {
        p.out_scores[out + i] = static_cast<float>(x.score);
        p.out_parents[out + i] = static_cast<int32_t>(row0 + x.beam);
        p.out_tokens[out + i] = static_cast<int32_t>(x.token);
    };
    uint32_t found = n;
    if (n > kRoom) {
        // too many that are nearly equal: the best one k times, each behind the last
        Candidate last = {INFINITY, 0, INFINITY, 0};
        found = 0;
        for (; found < p.k; ++found) {
            Candidate best = {-INFINITY, UINT_MAX, 0, UINT_MAX};
            for (uint32_t c = threadIdx.x; c < all; c += kThreads) {
                Candidate x;
                if (candidate(c, x) && better(last, x) && better(x, best)) best = x;
            }
            for (int i = 32; i; i >>= 1) {
                const Candidate o = {__shfl_xor(best.score, i), static_cast<uint32_t>(__shfl_xor(best.beam, i)), __shfl_xor(best.x, i),
                                     static_cast<uint32_t>(__shfl_xor(best.token, i))};
                if (better(o, best)) best = o;
            }
            __syncthreads();
            if (lane == 0) {
                s_score[wave] = best.score;
                s_beam[wave] = best.beam;
                s_x[wave] = best.x;
                s_token[wave] = best.token;
            }
            __syncthreads();
            for (uint32_t w = 0; w < kWaves; ++w) {
                const Candidate o = {s_score[w], s_beam[w], s_x[w], s_token[w]};
                if (better(o, best)) best = o;
            }
            if (best.beam == UINT_MAX) break;
            if (threadIdx.x == 0) write(found, best);
            last = best;
        }
    } else {
        for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
            const Candidate mine = {s_score[i], s_beam[i], s_x[i], s_token[i]};
            uint32_t rank = 0;
            for (uint32_t j = 0; j < n; ++j) rank += better(Candidate{s_score[j], s_beam[j], s_x[j], s_token[j]}, mine);
            if (rank < p.k) write(rank, mine);
        }
    }
    for (uint32_t i = found + threadIdx.x; i < p.k; i += kThreads) {
        p.out_scores[out + i] = -INFINITY;
        p.out_parents[out + i] = -1;
        p.out_tokens[out + i] = p.pad;
    }
}

// ---- Host -------------------------------------------------------------------

constexpr uint64_t kWantGroups = 8 * kComputeUnits;

struct Cut {
    uint32_t loads, part, parts;
};

// Parts as large as leave eight workgroups for each compute unit, of 1, 2, 4 or 8 loads.
Cut cut_of(uint64_t rows, uint64_t vocab) {
    Cut c = {8, 0, 0};
    while (c.loads > 1 && rows * ((vocab + c.loads * kThreads * kEach - 1) / (c.loads * kThreads * kEach)) < kWantGroups) c.loads /= 2;
    c.part = c.loads * kThreads * kEach;
    c.parts = static_cast<uint32_t>((vocab + c.part - 1) / c.part);
    return c;
}

bool sizes_ok(uint64_t batch, uint64_t beams, uint64_t vocab, uint32_t k) {
    if (k == 0 || k > kMaxK || beams == 0 || beams > kMaxBeams || vocab == 0 || vocab >= (uint64_t{1} << 31) / beams ||
        batch >= (uint64_t{1} << 24) / beams)
        return false;
    return batch * beams * cut_of(batch * beams, vocab).parts < (uint64_t{1} << 32) / kThreads;
}

uint64_t workspace_of(uint64_t rows, uint32_t parts, uint32_t k) { return rows * parts * (2 + 2 * uint64_t{k}) * sizeof(float); }

template <bool kF32>
auto part_kernel_of(uint32_t loads) {
    switch (loads) {
        case 8: return beam_part_kernel<kF32, 8>;
        case 4: return beam_part_kernel<kF32, 4>;
        case 2: return beam_part_kernel<kF32, 2>;
        default: return beam_part_kernel<kF32, 1>;
    }
}

df11_status select(const void *logits, uint32_t dtype, uint64_t batch, uint64_t beams, uint64_t vocab, uint64_t batch_stride,
                   uint64_t beam_stride, const float *scores, const uint8_t *done, uint32_t k, int32_t pad,
                   float *out_scores, int32_t *out_parents, int32_t *out_tokens, void *workspace, uint64_t workspace_bytes,
                   void *hip_stream) {
    if (dtype > DF11_LOGITS_FP32) return DF11_E_UNSUPPORTED;
    if (!sizes_ok(batch, beams, vocab, k) || batch_stride > kMaxStride || beam_stride > kMaxStride ||
        span(batch, batch_stride) + span(beams, beam_stride) >= kMaxExtent)
        return DF11_E_INVALID_ARG;
    if (batch == 0) return DF11_OK;
    const auto low = [](const void *x) { return reinterpret_cast<uintptr_t>(x); };
    if (!logits || !scores || !out_scores || !out_parents || !out_tokens || (low(logits) & (dtype == DF11_LOGITS_FP32 ? 3u : 1u)) ||
        ((low(scores) | low(out_scores) | low(out_parents) | low(out_tokens)) & 3u) || !aligned16(workspace))
        return DF11_E_INVALID_ARG;
    const uint64_t rows = batch * beams;
    const Cut cut = cut_of(rows, vocab);
    if (workspace_bytes < workspace_of(rows, cut.parts, k)) return DF11_E_BUFFER_TOO_SMALL;
    if (!workspace) return DF11_E_INVALID_ARG;
    BeamParams p;
    p.logits = logits;
    p.scores = scores;
    p.done = done;
    p.out_scores = out_scores;
    p.out_parents = out_parents;
    p.out_tokens = out_tokens;
    p.sums = static_cast<float *>(workspace);
    p.best = p.sums + rows * cut.parts * 2;
    p.at = reinterpret_cast<int32_t *>(p.best + rows * cut.parts * k);
    p.batch_stride = batch_stride;
    p.beam_stride = beam_stride;
    p.beams = static_cast<uint32_t>(beams);
    p.vocab = static_cast<uint32_t>(vocab);
    p.k = k;
    p.parts = cut.parts;
    p.part = cut.part;
    p.pad = pad;
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    auto fn = dtype == DF11_LOGITS_FP32 ? part_kernel_of<true>(cut.loads) : part_kernel_of<false>(cut.loads);
    hipError_t err = launch(fn, static_cast<uint32_t>(rows * cut.parts), kThreads, 0, st, p);
    if (err == hipSuccess) err = launch(beam_choose_kernel, static_cast<uint32_t>(batch), kThreads, 0, st, p);
    return launched(err);
}

}  // namespace

extern "C" uint64_t df11_beam_select_workspace_bytes(uint64_t batch, uint64_t beams, uint64_t vocab, uint32_t k) {
    if (!sizes_ok(batch, beams, vocab, k)) return 0;
    return workspace_of(batch * beams, cut_of(batch * beams, vocab).parts, k);
}

extern "C" df11_status df11_beam_select(const void *logits, uint32_t dtype, uint64_t batch, uint64_t beams, uint64_t vocab,
                                        uint64_t batch_stride, uint64_t beam_stride, const float *scores,
                                        const uint8_t *done, uint32_t k, int32_t pad, float *out_scores,
                                        int32_t *out_parents, int32_t *out_tokens, void *workspace,
                                        uint64_t workspace_bytes, void *hip_stream) {
    return df11i::guarded([&] {
        return select(logits, dtype, batch, beams, vocab, batch_stride, beam_stride, scores, done, k, pad, out_scores, out_parents,
                      out_tokens, workspace, workspace_bytes, hip_stream);
    });
}
