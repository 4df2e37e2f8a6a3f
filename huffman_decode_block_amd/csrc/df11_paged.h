// What the operators on the paged cache (include/df11_step.h,
// include/df11_search.h) share: where pages lie, conversions of what they hold,
// the checks of a cache on the host, launches.
#ifndef DF11_PAGED_H
#define DF11_PAGED_H

#include <hip/hip_runtime.h>

#include <algorithm>

#include "df11_internal.h"
#include "df11_step.h"
#include "df11_wave.h"

namespace df11p {

using df11w::v2u;
using df11w::v4u;

typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Pages {
    uint8_t *base;
    uint64_t page, head, row;  // strides in bytes
    const float *scale;
};

// Eight values that may start at any even address: the hardware loads them as
// they lie, without the compiler having to take them apart.
struct __attribute__((packed, aligned(2))) Eight {
    uint32_t w[4];
};

__device__ __forceinline__ v4u load8(const uint16_t *p) {
    const Eight t = *reinterpret_cast<const Eight *>(p);
    return v4u{t.w[0], t.w[1], t.w[2], t.w[3]};
}

// Two BF16 values from two bytes of E4M3 (exact).
template <bool kHigh>
__device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, kHigh));
}

__device__ __forceinline__ v4u from_e4m3x8(uint32_t a, uint32_t b) {
    return v4u{from_e4m3<false>(a), from_e4m3<true>(a), from_e4m3<false>(b), from_e4m3<true>(b)};
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    bf2 v;
    v.x = static_cast<__bf16>(a);
    v.y = static_cast<__bf16>(b);
    return __builtin_bit_cast(uint32_t, v);
}

// Two floats cut off to BF16.
__device__ __forceinline__ uint32_t cut2(float a, float b) {
    return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u);
}

// Two BF16 values that are not negative (or NaN), each held to at least the one in `least`.
__device__ __forceinline__ uint32_t at_least2(uint32_t v, uint32_t least) {
    typedef uint16_t u2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u2, v), __builtin_bit_cast(u2, least)));
}

constexpr uint32_t kLeastPart = 0x00800080u;  // twice 2^-126, the smallest normal number

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

constexpr uint32_t kMinPage = 8, kMaxPage = 1024;
constexpr uint32_t kComputeUnits = 256;

// ---- Host ------------------------------------------------------------------

template <class T>
struct Plain {
    typedef T type;
};

template <class... A>
hipError_t launch(void (*fn)(A...), uint32_t grid, uint32_t threads, uint32_t lds, hipStream_t st,
                  typename Plain<A>::type... a) {
    void *args[] = {&a...};
    return hipLaunchKernel(reinterpret_cast<const void *>(fn), dim3(grid), dim3(threads), args, lds, st);
}

inline df11_status launched(hipError_t err) {
    if (err == hipSuccess) return DF11_OK;
    df11i::last_hip_error = static_cast<int32_t>(err);
    return DF11_E_HIP;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool dim_ok(uint32_t d) { return d == 64 || d == 128 || d == 256; }

inline bool page_ok(uint32_t n) { return n >= kMinPage && n <= kMaxPage && (n & (n - 1)) == 0; }

constexpr uint64_t kMaxStride = uint64_t{1} << 40, kMaxExtent = uint64_t{1} << 48;  // elements

// What `n` steps of `stride` span, held to kMaxExtent; a few of these together
// are in bounds below that and cannot overflow.
inline uint64_t span(uint64_t n, uint64_t stride) { return n && stride > kMaxExtent / n ? kMaxExtent : n * stride; }

inline df11_status check_cache(const df11_paged_cache *c) {
    if (!c) return DF11_E_INVALID_ARG;
    if (c->dtype > DF11_CACHE_E4M3 || !dim_ok(c->head_dim) || !page_ok(c->page_size)) return DF11_E_UNSUPPORTED;
    if (!c->k_pages || !c->v_pages || !aligned16(c->k_pages) || !aligned16(c->v_pages)) return DF11_E_INVALID_ARG;
    if (c->kv_heads == 0 || c->kv_heads > 65536 || c->n_pages == 0 || c->n_pages > 0x7FFFFFFFu) return DF11_E_INVALID_ARG;
    const bool e4m3 = c->dtype == DF11_CACHE_E4M3;
    const uint64_t unit = e4m3 ? 16 : 8;  // elements in 16 bytes
    for (uint64_t s : {c->k_page_stride, c->k_head_stride, c->k_row_stride, c->v_page_stride, c->v_head_stride, c->v_row_stride})
        if (s % unit != 0 || s > kMaxStride) return DF11_E_INVALID_ARG;
    const auto extent = [&](uint64_t page, uint64_t head, uint64_t row) {
        return span(c->n_pages, page) + span(c->kv_heads, head) + span(c->page_size, row);
    };
    if (extent(c->k_page_stride, c->k_head_stride, c->k_row_stride) >= kMaxExtent ||
        extent(c->v_page_stride, c->v_head_stride, c->v_row_stride) >= kMaxExtent)
        return DF11_E_INVALID_ARG;
    if (e4m3 && (!c->k_scale || !c->v_scale)) return DF11_E_INVALID_ARG;
    return DF11_OK;
}

inline uint32_t log2_of(uint32_t v) { return 31u - static_cast<uint32_t>(__builtin_clz(v)); }

inline Pages k_of(const df11_paged_cache *c) {
    const uint64_t e = c->dtype == DF11_CACHE_E4M3 ? 1 : 2;
    return Pages{static_cast<uint8_t *>(c->k_pages), c->k_page_stride * e, c->k_head_stride * e, c->k_row_stride * e, c->k_scale};
}

inline Pages v_of(const df11_paged_cache *c) {
    const uint64_t e = c->dtype == DF11_CACHE_E4M3 ? 1 : 2;
    return Pages{static_cast<uint8_t *>(c->v_pages), c->v_page_stride * e, c->v_head_stride * e, c->v_row_stride * e, c->v_scale};
}

}  // namespace df11p

#endif  // DF11_PAGED_H
