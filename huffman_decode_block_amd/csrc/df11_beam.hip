// Selection of a beam search (gfx950): the best continuations of each search's
// beams over a vocabulary (include/df11_search.h).
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>

#include "df11_paged.h"
#include "df11_search.h"

namespace {

using namespace df11p;

// A beam's continuation scores s + x - log sum exp(x): the k best of a part of the
// logits are among the parts' k best whatever the sum is, so that one pass over the
// logits is enough.  Two kernels.  In the first a workgroup takes a part of a beam's
// logits into registers, whole: their maximum, their sum of exponentials, and the k
// best.  The second adds the parts' sums to each beam's logarithm, in 64 bits, and
// chooses among all parts' best ones.
//
// 32 searches of 8 beams over 128,256 BF16 logits, 16 chosen (52 MB of beams that
// go on): 20 us for the first kernel, 8.8 for the second.  The first is bound by its workgroups' chains
// (load, maxima, threshold, ranks: two rounds of four on a compute unit), 2.6 TB/s.
// One search of 4 beams over 32,000: 4.4 + 5.0, a kernel's start and end and one chain
// each; of 16 beams over 160,000, the best 32: 9.3 + 16.5, 40,448 candidates in one workgroup.
//
// Choosing k of n: with t the k-th largest of the largest values of 256 sets, at least
// k values reach t, and few more do if the largest ones are spread over the sets; they
// go to LDS in any order, and each counts those before it (eight at a time: one at a time
// the reads from LDS, each waited for, were a third of both kernels).  t is sought bit
// by bit, some of the bits (a value that is lower than the k-th largest only lets more
// values through).  Only where more values than LDS has room for are equal, or nearly so,
// are the best sought one after the other.  The sets are the threads' values in the first
// kernel; of one wave's lanes the 64th largest value is the smallest, which too many
// reach.  In the second a list's places go to different sets: as they lie,
// a thread would have one place of each list where k divides 256, its best or its worst
// (16 beams over 160,000: k = 32 1,896 us in place of 27, 64 7,346 in place of 48).

constexpr uint32_t kThreads = 256, kWaves = kThreads / 64;
constexpr uint32_t kMaxK = 64;
constexpr uint32_t kRoom = 1024;  // values that may reach t before they are sought one by one
constexpr uint32_t kEach = 8;     // values of a load
constexpr uint32_t kAtOnce = 8;   // values compared with one: their reads from LDS overlap

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

constexpr uint32_t kTops = 256;  // values among which the k-th largest is sought

// Of the keys of kTops values, in LDS, kPer in each lane: the largest of groups.
template <int kPer, int kBits>
__device__ __forceinline__ float reached(const uint32_t *keys, uint32_t k) {
    uint32_t key[kPer] = {};
#pragma unroll
    for (uint32_t i = 0; i < kTops / 64; ++i) key[i % kPer] = max(key[i % kPer], keys[i * 64 + (threadIdx.x & 63u)]);
    const auto reaching = [&](uint32_t t) {
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) n += __popcll(__ballot(key[i] >= t));
        return n;
    };
    uint32_t t = 0;
#pragma unroll
    for (int bit = 31; bit > 31 - kBits; --bit) {
        const uint32_t with = t | 1u << bit;
        if (reaching(with) >= k) t = with;
    }
    return fmaxf(of_key(t), -INFINITY);  // NaN for keys below that of -infinity
}

// A value that at least k of them reach (-infinity where fewer are more), near the k-th
// largest: kBits of it.  Groups as large as leave four for each of the k.
template <int kBits>
__device__ __forceinline__ float reached_by(const uint32_t *keys, uint32_t k) {
    return k <= kTops / 16 ? reached<1, kBits>(keys, k) : k <= kTops / 8 ? reached<2, kBits>(keys, k) : reached<4, kBits>(keys, k);
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

// Eight tokens' logits as they are in memory: BF16 takes half of the registers.
template <bool kF32>
struct Eight {
    uint32_t w[kF32 ? 8 : 4];
    __device__ __forceinline__ float operator[](int j) const {
        if (kF32) return __builtin_bit_cast(float, w[j % (kF32 ? 8 : 4)]);
        return __builtin_bit_cast(float, j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
    }
};

// Those from `at` on; -infinity from `end` on.
template <bool kF32>
__device__ __forceinline__ Eight<kF32> load_logits(const void *row, uint32_t at, uint32_t end) {
    Eight<kF32> x;
    if (at + kEach <= end) {
        if (kF32) {
            const EightFloats w = *reinterpret_cast<const EightFloats *>(static_cast<const float *>(row) + at);
#pragma unroll
            for (int i = 0; i < (kF32 ? 8 : 4); ++i) x.w[i] = __builtin_bit_cast(uint32_t, w.x[i]);
        } else {
            const v4u w = load8(static_cast<const uint16_t *>(row) + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) x.w[i] = w[i];
        }
    } else if (kF32) {
#pragma unroll
        for (int i = 0; i < (kF32 ? 8 : 4); ++i)
            x.w[i] = at + i < end ? static_cast<const uint32_t *>(row)[at + i] : 0xFF800000u;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint16_t *from = static_cast<const uint16_t *>(row) + at + 2 * i;
            x.w[i] = (at + 2 * i < end ? from[0] : 0xFF80u) | (at + 2 * i + 1 < end ? from[1] : 0xFF80u) << 16;
        }
    }
    return x;
}

template <bool kF32, int kLoads>
__global__ void __launch_bounds__(kThreads) beam_part_kernel(BeamParams p) {
    __shared__ float s_max[kWaves], s_sum[kWaves];
    __shared__ uint32_t s_top[kTops];
    __shared__ __attribute__((aligned(16))) float s_x[kRoom + kAtOnce];
    __shared__ __attribute__((aligned(16))) uint32_t s_at[kRoom + kAtOnce];
    __shared__ uint32_t s_n;
    const uint32_t row = blockIdx.x / p.parts, part = blockIdx.x - row * p.parts;
    const float score = p.scores[row];
    const bool done = p.done && p.done[row];
    if (done || !(fabsf(score) < INFINITY)) return;
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t b = row / p.beams;
    const uint64_t first = b * p.batch_stride + (row - b * p.beams) * p.beam_stride;
    const void *logits = static_cast<const uint8_t *>(p.logits) + first * (kF32 ? 4 : 2);
    const uint32_t begin = part * p.part, end = min(begin + p.part, p.vocab);

    Eight<kF32> x[kLoads];
    const auto token = [&](int i, int j) { return begin + (i * kThreads + threadIdx.x) * kEach + j; };
#pragma unroll
    for (int i = 0; i < kLoads; ++i) x[i] = load_logits<kF32>(logits, token(i, 0), end);
    float top = -INFINITY, tops[kLoads];  // NaN aside, which makes the sum NaN
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        tops[i] = x[i][0];
#pragma unroll
        for (int j = 1; j < static_cast<int>(kEach); ++j) tops[i] = fmaxf(tops[i], x[i][j]);
        top = fmaxf(top, tops[i]);
    }
    const float wave_top = wave_max(top);
    static_assert(kTops == kThreads, "each thread's largest");
    s_top[threadIdx.x] = key_of(top);
    if (lane == 0) s_max[wave] = wave_top;
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    const float t = reached_by<16>(s_top, p.k);
    float m = s_max[0];
#pragma unroll
    for (uint32_t w = 1; w < kWaves; ++w) m = fmaxf(m, s_max[w]);
    // unpacked anew each time: kept, the floats would take twice the registers
    const auto as_loaded = [&] {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (uint32_t &w : x[i].w) asm volatile("" : "+v"(w));
    };
    as_loaded();
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
    as_loaded();

    // values that reach t: most loads have none in a whole wave
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        if (!__any(tops[i] >= t)) continue;
#pragma unroll
        for (int j = 0; j < static_cast<int>(kEach); ++j)
            if (x[i][j] >= t && x[i][j] > -INFINITY) {
                const uint32_t n = atomicAdd(&s_n, 1u);
                if (n < kRoom) {
                    s_x[n] = x[i][j];
                    s_at[n] = token(i, j);
                }
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
            as_loaded();
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
    if (threadIdx.x < kAtOnce) s_x[n + threadIdx.x] = -INFINITY;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
        const float v = s_x[i];
        const uint32_t at = s_at[i];
        uint32_t rank = 0;
        for (uint32_t j = 0; j < n; j += kAtOnce) {
#pragma unroll
            for (uint32_t e = 0; e < kAtOnce; e += 4) {
                const f4 o = *reinterpret_cast<const f4 *>(&s_x[j + e]);
                const v4u o_at = *reinterpret_cast<const v4u *>(&s_at[j + e]);
#pragma unroll
                for (int k = 0; k < 4; ++k) rank += (o[k] > v) | ((o[k] == v) & (o_at[k] < at));
            }
        }
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
    // without branches: ties are common among BF16 logits
    const bool token = a.token < b.token, x = (a.x > b.x) | ((a.x == b.x) & token);
    const bool beam = (a.beam < b.beam) | ((a.beam == b.beam) & x);
    return (a.score > b.score) | ((a.score == b.score) & beam);
}

constexpr uint32_t kMaxBeams = 1024;
constexpr uint32_t kHeld = 4;  // candidates that a thread holds in registers

__global__ void __launch_bounds__(kThreads) beam_choose_kernel(BeamParams p) {
    __shared__ double s_lse[kMaxBeams];  // NaN for a beam that offers no token
    __shared__ float s_from[kMaxBeams];  // the beams' scores
    __shared__ uint8_t s_done[kMaxBeams];
    __shared__ __attribute__((aligned(16))) double s_score[kRoom + kAtOnce];
    __shared__ __attribute__((aligned(16))) float s_x[kRoom + kAtOnce];
    __shared__ __attribute__((aligned(16))) uint32_t s_beam[kRoom + kAtOnce], s_token[kRoom + kAtOnce];
    __shared__ uint32_t s_top[2][kTops];
    __shared__ uint32_t s_list[kRoom];
    __shared__ uint32_t s_n, s_lists;
    const uint32_t b = blockIdx.x, lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint64_t row0 = uint64_t{b} * p.beams;

    // candidate c: place c % k of list c / k, a part of a beam, best first; a beam that
    // has ended has one, its first.  All of them, or the first of each list, are on
    // their way while the beams' sums are added; what a beam without tokens has there is
    // not looked at.
    const uint32_t lists = p.parts * p.beams, per_beam = p.parts * p.k, all = lists * p.k;
    const bool few = all <= kHeld * kThreads;
    float held_x[kHeld];
    int32_t held_at[kHeld];
#pragma unroll
    for (uint32_t h = 0; h < kHeld; ++h) {
        const uint32_t i = h * kThreads + threadIdx.x, c = few ? min(i, all - 1) : min(i, lists - 1) * p.k;
        held_x[h] = p.best[row0 * per_beam + c];
        held_at[h] = p.at[row0 * per_beam + c];
    }
    // as many lanes for a beam as there are, a power of two
    const uint32_t share = min(64u, kThreads >> (32 - __builtin_clz(min(p.beams, kThreads) * 2 - 1) - 1)), mine = threadIdx.x % share;
    for (uint32_t i0 = 0; i0 < p.beams; i0 += kThreads / share) {
        const uint32_t i = i0 + threadIdx.x / share;
        const uint64_t row = row0 + min(i, p.beams - 1);
        const v2f *sums = reinterpret_cast<const v2f *>(p.sums) + row * p.parts;
        v2f s[2];  // the first of a lane's parts
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) s[h] = sums[min(mine + h * share, p.parts - 1)];
        const float from = p.scores[row];
        const bool done = p.done && p.done[row];
        float m = -INFINITY;
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h)
            if (mine + h * share < p.parts) m = fmaxf(m, s[h].x);
        for (uint32_t c = mine + 2 * share; c < p.parts; c += share) m = fmaxf(m, sums[c].x);
        for (uint32_t k = share / 2; k; k >>= 1) m = fmaxf(m, __shfl_xor(m, k));
        const auto part = [&](v2f x) {
            return x.x == -INFINITY ? static_cast<double>(x.y != x.y ? NAN : 0.0f)
                                    : static_cast<double>(x.y) * exp(static_cast<double>(x.x) - static_cast<double>(m));
        };
        double sum = 0;
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h)
            if (mine + h * share < p.parts) sum += part(s[h]);
        for (uint32_t c = mine + 2 * share; c < p.parts; c += share) sum += part(sums[c]);
        for (uint32_t k = share / 2; k; k >>= 1) sum += __shfl_xor(sum, k);
        if (mine == 0 && i < p.beams) {
            s_lse[i] = done || !(fabsf(from) < INFINITY) ? static_cast<double>(NAN) : static_cast<double>(m) + log(sum);
            s_from[i] = from;
            s_done[i] = done;
        }
    }
    s_top[0][threadIdx.x] = s_top[1][threadIdx.x] = key_of(-INFINITY);
    if (threadIdx.x == 0) s_n = s_lists = 0;
    __syncthreads();

    const auto of = [&](uint32_t c, float x, int32_t token, Candidate &out) {
        const uint32_t beam = c / per_beam;
        out.beam = beam;
        if (s_done[beam]) {
            out.score = s_from[beam];
            out.x = 0;
            out.token = static_cast<uint32_t>(p.pad);
            return c == beam * per_beam && fabsf(s_from[beam]) < INFINITY;
        }
        const double lse = s_lse[beam];
        out.x = x;
        out.token = static_cast<uint32_t>(token);
        out.score = static_cast<double>(s_from[beam]) + (static_cast<double>(x) - lse);
        return fabs(lse) < INFINITY && x > -INFINITY;
    };
    const auto candidate = [&](uint32_t c, Candidate &out) {
        const uint64_t at = row0 * per_beam + c;
        return of(c, p.best[at], p.at[at], out);
    };
    const auto show = [&](uint32_t *tops, uint32_t at, double score) {
        if (score > -INFINITY) atomicMax(&tops[at % kTops], key_of(static_cast<float>(score)));
    };
    // Of many lists those that may hold one of the k best: their first ones reach the
    // k-th largest of all lists'.  Where more do than LDS names, all are looked at.
    uint32_t there = lists;
    bool named = false;
    if (!few) {
        float first[kHeld];
#pragma unroll
        for (uint32_t h = 0; h < kHeld; ++h) {
            const uint32_t list = h * kThreads + threadIdx.x;
            Candidate x;
            first[h] = list < lists && of(list * p.k, held_x[h], held_at[h], x) ? static_cast<float>(x.score) : NAN;
            show(s_top[0], list, first[h]);
        }
        for (uint32_t list = kHeld * kThreads + threadIdx.x; list < lists; list += kThreads) {
            Candidate x;
            if (candidate(list * p.k, x)) show(s_top[0], list, x.score);
        }
        __syncthreads();
        const float least = reached_by<20>(s_top[0], p.k);
        const auto note = [&](uint32_t list) {
            const uint32_t n = atomicAdd(&s_lists, 1u);
            if (n < kRoom) s_list[n] = list;
        };
#pragma unroll
        for (uint32_t h = 0; h < kHeld; ++h)
            if (first[h] >= least) note(h * kThreads + threadIdx.x);
        for (uint32_t list = kHeld * kThreads + threadIdx.x; list < lists; list += kThreads) {
            Candidate x;
            if (candidate(list * p.k, x) && static_cast<float>(x.score) >= least) note(list);
        }
        __syncthreads();
        named = s_lists <= kRoom;
        if (named) there = s_lists;
    }
    // Those lists' candidates: at least k of them reach the k-th largest of the largest
    // in kTops sets, and few more.  Places of one list, and lists at one place, are of
    // different sets.
    const uint32_t size = there * p.k, apart = there | 1;
    const bool fit = size <= kHeld * kThreads;
    const auto place = [&](uint32_t i) { return named ? s_list[i / p.k] * p.k + i % p.k : i; };
    if (named && fit && size) {
#pragma unroll
        for (uint32_t h = 0; h < kHeld; ++h) {
            const uint64_t at = row0 * per_beam + place(min(h * kThreads + threadIdx.x, size - 1));
            held_x[h] = p.best[at];
            held_at[h] = p.at[at];
        }
    }
    Candidate held[kHeld];
#pragma unroll
    for (uint32_t h = 0; h < kHeld; ++h) {
        const uint32_t i = h * kThreads + threadIdx.x;
        if (!fit || i >= size || !of(place(i), held_x[h], held_at[h], held[h])) held[h].score = -INFINITY;
        show(s_top[1], i / p.k + i % p.k * apart, held[h].score);
    }
    if (!fit)
        for (uint32_t i = threadIdx.x; i < size; i += kThreads) {
            Candidate x;
            if (candidate(place(i), x)) show(s_top[1], i / p.k + i % p.k * apart, x.score);
        }
    __syncthreads();
    const float t = reached_by<20>(s_top[1], p.k);
    const auto keep = [&](const Candidate &x) {
        const uint32_t n = atomicAdd(&s_n, 1u);
        if (n < kRoom) {
            s_score[n] = x.score;
            s_beam[n] = x.beam;
            s_x[n] = x.x;
            s_token[n] = x.token;
        }
    };
#pragma unroll
    for (uint32_t h = 0; h < kHeld; ++h)
        if (held[h].score > -INFINITY && static_cast<float>(held[h].score) >= t) keep(held[h]);
    if (!fit)
        for (uint32_t i = threadIdx.x; i < size; i += kThreads) {
            Candidate x;
            if (candidate(place(i), x) && static_cast<float>(x.score) >= t) keep(x);
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
        if (threadIdx.x < kAtOnce) s_score[n + threadIdx.x] = -INFINITY;
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
            const Candidate mine = {s_score[i], s_beam[i], s_x[i], s_token[i]};
            uint32_t rank = 0;
            for (uint32_t j = 0; j < n; j += kAtOnce)
#pragma unroll
                for (uint32_t e = 0; e < kAtOnce; ++e)
                    rank += better(Candidate{s_score[j + e], s_beam[j + e], s_x[j + e], s_token[j + e]}, mine);
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
// A large part pays once for its threshold and ranks and gives the second kernel fewer
// candidates.  32 x 8 beams over 128,256 take 28.4 us so, with sixteen for each 27.9,
// with four 28.6; 8 x 4 beams, the best 8, 15.5, 15.2 and 13.5.
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
