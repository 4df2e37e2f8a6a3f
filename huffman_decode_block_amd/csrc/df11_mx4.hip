// 4-bit weights (gfx950): quantisation, expansion to BF16, and the product of
// BF16 activations with them (include/df11_step.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "df11_internal.h"
#include "df11_step.h"
#include "df11_wave.h"

namespace {

using df11w::kOff;
using df11w::rsrc;
using df11w::Rsrc;
using df11w::v2u;
using df11w::v4u;

typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr uint64_t kMaxCols = uint64_t{1} << 24;    // columns and strides: a tile's byte offsets fit 32 bits
constexpr uint64_t kMaxValues = uint64_t{1} << 40;  // values of one matrix
constexpr uint32_t kBlock = 32;                     // values that share a scale
constexpr uint32_t kNanScale = 255;

// ---- Quantisation ----------------------------------------------------------
// Four lanes take one block of 32 values, 8 values (16 bytes) each; the
// block's maximum goes round the four by two DPP exchanges.  Bound by HBM: 2
// bytes read and 17/32 written for a value.  An item is a block; items are
// numbered row by row, so that rows of any width fill the lanes.

constexpr uint32_t kQuantThreads = 256;
constexpr uint32_t kQuantItems = kQuantThreads / 4;  // blocks per workgroup and step

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    const uint32_t a = __builtin_amdgcn_update_dpp(0u, v, 0xB1, 0xF, 0xF, true);  // lanes 1 0 3 2
    v = v > a ? v : a;
    const uint32_t b = __builtin_amdgcn_update_dpp(0u, v, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
    return v > b ? v : b;
}

template <bool kAligned>
__global__ void __launch_bounds__(kQuantThreads)
quantize_kernel(const uint16_t *x, uint64_t row_stride, uint32_t cols, uint32_t blocks, uint64_t items,
                uint8_t *codes, uint8_t *scales) {
    const uint32_t part = threadIdx.x & 3u;
    for (uint64_t base = uint64_t{blockIdx.x} * kQuantItems; base < items; base += uint64_t{gridDim.x} * kQuantItems) {
        const uint64_t row0 = base / blocks;  // uniform
        const uint32_t local = static_cast<uint32_t>(base - row0 * blocks) + (threadIdx.x >> 2);
        const uint64_t item = base + (threadIdx.x >> 2);
        if (item >= items) continue;  // whole quads
        const uint32_t down = local / blocks, block = local - down * blocks;
        const uint64_t row = row0 + down;
        const uint32_t col = block * kBlock + part * 8;
        const uint16_t *src = x + row * row_stride + col;
        uint32_t w[4];  // two values each
        if (kAligned && col + 8 <= cols) {
            const v4u t = *reinterpret_cast<const v4u *>(src);
            w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                const uint32_t lo = col + 2 * i < cols ? src[2 * i] : 0u;
                const uint32_t hi = col + 2 * i + 1 < cols ? src[2 * i + 1] : 0u;
                w[i] = lo | (hi << 16);
            }
        }
        // magnitudes of BF16 compare like their bits, infinities and NaN above all
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
            top = lo > top ? lo : top;
            top = hi > top ? hi : top;
        }
        top = quad_max(top);
        // floor(log2 a) + 127 is the exponent field; of a denormal it is 126
        // or more below, which the lower limit of e hides
        const uint32_t field = top >> 7;
        const uint32_t s = field > 2 ? field - 2 : 0;
        const bool bad = field == 255;
        // 2^-e = 2^(127 - s): s <= 252, so the field 254 - s is a normal number's
        const float inv = __builtin_bit_cast(float, (254u - s) << 23);
        uint32_t code = 0;
        {
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __builtin_bit_cast(float, w[i] << 16) * inv;
                v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u) * inv;
            }
            code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[0], v[1], 1.0f, 0);
            code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[2], v[3], 1.0f, 1);
            code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[4], v[5], 1.0f, 2);
            code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[6], v[7], 1.0f, 3);
        }
        if (bad) code = 0;
        *reinterpret_cast<uint32_t *>(codes + item * 16 + part * 4) = code;
        if (part == 0) scales[item] = static_cast<uint8_t>(bad ? kNanScale : s);
    }
}

// ---- Expansion to BF16 -----------------------------------------------------

// Two BF16 values of one byte of codes under scale byte s; the conversion
// takes the scale as a 32-bit float of which it reads the exponent.
template <int kByte>
__device__ __forceinline__ uint32_t expand2(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, kByte));
}

__device__ __forceinline__ v4u expand8(uint32_t codes, float scale) {
    return v4u{expand2<0>(codes, scale), expand2<1>(codes, scale), expand2<2>(codes, scale), expand2<3>(codes, scale)};
}

template <bool kAligned>
__global__ void __launch_bounds__(kQuantThreads)
dequantize_kernel(const uint8_t *codes, const uint8_t *scales, uint32_t cols, uint32_t blocks, uint64_t items,
                  uint16_t *out, uint64_t out_stride) {
    const uint32_t part = threadIdx.x & 3u;
    for (uint64_t base = uint64_t{blockIdx.x} * kQuantItems; base < items; base += uint64_t{gridDim.x} * kQuantItems) {
        const uint64_t row0 = base / blocks;
        const uint32_t local = static_cast<uint32_t>(base - row0 * blocks) + (threadIdx.x >> 2);
        const uint64_t item = base + (threadIdx.x >> 2);
        if (item >= items) continue;
        const uint32_t down = local / blocks, block = local - down * blocks;
        const uint64_t row = row0 + down;
        const uint32_t col = block * kBlock + part * 8;
        const uint32_t code = *reinterpret_cast<const uint32_t *>(codes + item * 16 + part * 4);
        const uint32_t s = scales[item];
        v4u o = expand8(code, __builtin_bit_cast(float, s << 23));
        if (s == kNanScale) o = v4u{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
        uint16_t *dst = out + row * out_stride + col;
        if (kAligned && col + 8 <= cols) {
            *reinterpret_cast<v4u *>(dst) = o;
        } else {
            const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i)
                if (col + i < cols) dst[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
        }
    }
}

// ---- Product ---------------------------------------------------------------

// Copies x into rows of `width` values (a multiple of 32), zeros past k: what
// the product reads where x itself cannot be read 16 bytes at a time.
__global__ void __launch_bounds__(256)
pack_rows_kernel(const uint16_t *x, uint64_t x_stride, uint32_t k, uint32_t width, uint64_t m, uint16_t *to) {
    const uint64_t total = m * (width / 8);
    for (uint64_t i = uint64_t{blockIdx.x} * 256 + threadIdx.x; i < total; i += uint64_t{gridDim.x} * 256) {
        const uint64_t row = i / (width / 8);
        const uint32_t col = static_cast<uint32_t>(i - row * (width / 8)) * 8;
        const uint16_t *src = x + row * x_stride + col;
        uint32_t w[4];
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t lo = col + 2 * j < k ? src[2 * j] : 0u;
            const uint32_t hi = col + 2 * j + 1 < k ? src[2 * j + 1] : 0u;
            w[j] = lo | (hi << 16);
        }
        *reinterpret_cast<v4u *>(to + 8 * i) = v4u{w[0], w[1], w[2], w[3]};
    }
}

struct MulParams {
    const uint16_t *x;
    const uint8_t *codes, *scales;
    uint16_t *y;
    uint64_t x_stride, y_stride;
    uint32_t m, n, blocks;  // blocks of 32 along k
};

// Token form: a workgroup takes 16 rows of w, its waves share k between them
// and add their sums in LDS.  A lane reads 16 bytes of codes at a time, which
// is one block of one row: lane l has row l % 16 and block 4 s + l / 16 of
// step s.  The matrix instruction's k index is ours to choose, as long as both
// operands agree: its i-th instruction of a step takes codes 8 i .. 8 i + 7 of
// every lane's block, so nothing moves between lanes and one scale serves all
// of a lane's codes.
constexpr uint32_t kTokenWaves = 8;

template <int kTiles>  // tiles of 16 rows of x
__global__ void __launch_bounds__(64 * kTokenWaves)
token_kernel(MulParams p) {
    __shared__ float s_sum[kTokenWaves][16 * 16];
    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * kTiles;
    const uint32_t rows_n = min(16u, p.n - n0);
    const Rsrc wr = rsrc(p.codes + uint64_t{n0} * p.blocks * 16, rows_n * p.blocks * 16);
    const Rsrc sr = rsrc(p.scales + uint64_t{n0} * p.blocks, rows_n * p.blocks);
    f4 acc[kTiles] = {};
    const uint32_t steps = (p.blocks + 3) / 4;
    for (uint32_t s = wave; s < steps; s += kTokenWaves) {
        const uint32_t block = 4 * s + q;
        const bool in = block < p.blocks;
        const v4u c = __builtin_amdgcn_raw_buffer_load_b128(wr, in ? (r * p.blocks + block) * 16 : kOff, 0, 0);
        const uint32_t sb = __builtin_amdgcn_raw_buffer_load_b8(sr, in ? r * p.blocks + block : kOff, 0, 0);
        const float scale = __builtin_bit_cast(float, (sb & 255u) << 23);
        const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
        bf8 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(bf8, expand8(cw[i], scale));
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const uint32_t row = m0 + 16 * t + r;
            const bool live = in && row < p.m;
            const v4u *src = reinterpret_cast<const v4u *>(p.x + uint64_t{row} * p.x_stride + block * kBlock);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const v4u xv = live ? src[i] : v4u{0, 0, 0, 0};
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], __builtin_bit_cast(bf8, xv), acc[t], 0, 0, 0);
            }
        }
    }
    // acc: column lane % 16 (a row of x), rows 4 (lane / 16) + 0..3 (of w)
    for (int t = 0; t < kTiles; ++t) {
        __syncthreads();
        *reinterpret_cast<f4 *>(&s_sum[wave][r * 16 + 4 * q]) = acc[t];
        __syncthreads();
        if (threadIdx.x < 256) {
            const uint32_t row = m0 + 16 * t + threadIdx.x / 16, col = n0 + threadIdx.x % 16;
            float v = 0;
            for (uint32_t k = 0; k < kTokenWaves; ++k) v += s_sum[k][threadIdx.x];
            if (row < p.m && col < p.n)
                p.y[uint64_t{row} * p.y_stride + col] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
        }
    }
}

// ---- Host ------------------------------------------------------------------

df11_status launched(hipError_t err) {
    if (err == hipSuccess) return DF11_OK;
    df11i::last_hip_error = static_cast<int32_t>(err);
    return DF11_E_HIP;
}

template <class T>
struct Plain {
    typedef T type;
};

template <class... A>
hipError_t launch(void (*fn)(A...), dim3 grid, uint32_t threads, hipStream_t st, typename Plain<A>::type... a) {
    void *args[] = {&a...};
    return hipLaunchKernel(reinterpret_cast<const void *>(fn), grid, dim3(threads), args, 0, st);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool matrix_ok(uint64_t rows, uint64_t cols, uint64_t stride) {
    return cols > 0 && cols <= kMaxCols && rows <= kMaxValues / cols && stride >= cols &&
           (rows == 0 || stride <= (uint64_t{1} << 48) / rows);
}

uint32_t quant_grid(uint64_t items) {
    return static_cast<uint32_t>(std::min<uint64_t>((items + kQuantItems - 1) / kQuantItems, 1u << 20));
}

df11_status quantize(const uint16_t *x, uint64_t rows, uint64_t cols, uint64_t row_stride, uint8_t *codes,
                     uint8_t *scales, void *hip_stream) {
    if (!matrix_ok(rows, cols, row_stride)) return DF11_E_INVALID_ARG;
    if (rows == 0) return DF11_OK;
    if (!x || !codes || !scales || !aligned16(codes) || (reinterpret_cast<uintptr_t>(x) & 1u)) return DF11_E_INVALID_ARG;
    const uint32_t blocks = static_cast<uint32_t>((cols + kBlock - 1) / kBlock);
    const uint64_t items = rows * blocks;
    const bool al = aligned16(x) && row_stride % 8 == 0;
    return launched(launch(al ? quantize_kernel<true> : quantize_kernel<false>, dim3(quant_grid(items)), kQuantThreads,
                           static_cast<hipStream_t>(hip_stream), x, row_stride, static_cast<uint32_t>(cols), blocks,
                           items, codes, scales));
}

df11_status dequantize(const uint8_t *codes, const uint8_t *scales, uint64_t rows, uint64_t cols, uint16_t *out,
                       uint64_t out_stride, void *hip_stream) {
    if (!matrix_ok(rows, cols, out_stride)) return DF11_E_INVALID_ARG;
    if (rows == 0) return DF11_OK;
    if (!out || !codes || !scales || !aligned16(codes) || (reinterpret_cast<uintptr_t>(out) & 1u))
        return DF11_E_INVALID_ARG;
    const uint32_t blocks = static_cast<uint32_t>((cols + kBlock - 1) / kBlock);
    const uint64_t items = rows * blocks;
    const bool al = aligned16(out) && out_stride % 8 == 0;
    return launched(launch(al ? dequantize_kernel<true> : dequantize_kernel<false>, dim3(quant_grid(items)),
                           kQuantThreads, static_cast<hipStream_t>(hip_stream), codes, scales,
                           static_cast<uint32_t>(cols), blocks, items, out, out_stride));
}

// Rows of x are read 16 bytes at a time and whole blocks at a time: anything
// else goes through a packed copy in the workspace.
bool needs_copy(uint64_t k, bool x_aligned) { return !x_aligned || k % kBlock != 0; }

uint64_t copy_bytes(uint64_t m, uint64_t k) { return m * ((k + kBlock - 1) / kBlock) * kBlock * 2; }

uint64_t matmul_workspace(uint64_t m, uint64_t n, uint64_t k, bool x_aligned) {
    (void)n;
    return needs_copy(k, x_aligned) ? copy_bytes(m, k) : 0;
}

df11_status matmul(const uint16_t *x, uint64_t m, uint64_t k, uint64_t x_stride, const uint8_t *codes,
                   const uint8_t *scales, uint64_t n, uint16_t *y, uint64_t y_stride, void *workspace,
                   uint64_t workspace_bytes, void *hip_stream) {
    if (m > 0x7FFFFFFFu || n > 0x7FFFFFFFu || k > kMaxCols || x_stride > kMaxCols || x_stride < k || y_stride < n)
        return DF11_E_INVALID_ARG;
    if (m == 0 || n == 0) return DF11_OK;
    if (!y || (k && (!x || !codes || !scales)) || !aligned16(codes) || (reinterpret_cast<uintptr_t>(x) & 1u) ||
        (reinterpret_cast<uintptr_t>(y) & 1u) || (workspace && !aligned16(workspace)))
        return DF11_E_INVALID_ARG;
    const bool al = aligned16(x) && x_stride % 8 == 0;
    if (workspace_bytes < matmul_workspace(m, n, k, al)) return DF11_E_BUFFER_TOO_SMALL;
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    MulParams p;
    p.x = x;
    p.codes = codes;
    p.scales = scales;
    p.y = y;
    p.x_stride = x_stride;
    p.y_stride = y_stride;
    p.m = static_cast<uint32_t>(m);
    p.n = static_cast<uint32_t>(n);
    p.blocks = static_cast<uint32_t>((k + kBlock - 1) / kBlock);
    hipError_t err = hipSuccess;
    if (needs_copy(k, al)) {
        if (!workspace) return DF11_E_INVALID_ARG;
        const uint32_t width = p.blocks * kBlock;
        const uint64_t lanes = m * (width / 8);
        if (lanes)
            err = launch(pack_rows_kernel, dim3(static_cast<uint32_t>(std::min<uint64_t>((lanes + 255) / 256, 8192))), 256,
                         st, x, x_stride, static_cast<uint32_t>(k), width, m, static_cast<uint16_t *>(workspace));
        if (err != hipSuccess) return launched(err);
        p.x = static_cast<const uint16_t *>(workspace);
        p.x_stride = width;
    }
    const uint32_t gn = static_cast<uint32_t>((n + 15) / 16);
    if (m <= 16)
        err = launch(token_kernel<1>, dim3(gn, 1), 64 * kTokenWaves, st, p);
    else
        err = launch(token_kernel<4>, dim3(gn, static_cast<uint32_t>((m + 63) / 64)), 64 * kTokenWaves, st, p);
    return launched(err);
}

}  // namespace

extern "C" df11_status df11_mx4_quantize(const uint16_t *x, uint64_t rows, uint64_t cols, uint64_t row_stride,
                                         uint8_t *codes, uint8_t *scales, void *hip_stream) {
    return df11i::guarded([&] { return quantize(x, rows, cols, row_stride, codes, scales, hip_stream); });
}

extern "C" df11_status df11_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, uint64_t rows, uint64_t cols,
                                           uint16_t *out, uint64_t out_stride, void *hip_stream) {
    return df11i::guarded([&] { return dequantize(codes, scales, rows, cols, out, out_stride, hip_stream); });
}

extern "C" uint64_t df11_mx4_matmul_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, int32_t x_aligned) {
    if (m > 0x7FFFFFFFu || n > 0x7FFFFFFFu || k > kMaxCols) return 0;  // refused by the product
    return matmul_workspace(m, n, k, x_aligned != 0);
}

extern "C" df11_status df11_mx4_matmul(const uint16_t *x, uint64_t m, uint64_t k, uint64_t x_stride,
                                       const uint8_t *codes, const uint8_t *scales, uint64_t n, uint16_t *y,
                                       uint64_t y_stride, void *workspace, uint64_t workspace_bytes,
                                       void *hip_stream) {
    return df11i::guarded([&] {
        return matmul(x, m, k, x_stride, codes, scales, n, y, y_stride, workspace, workspace_bytes, hip_stream);
    });
}
