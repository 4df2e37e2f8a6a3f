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

constexpr uint64_t kMaxCols = uint64_t{1} << 24;    // columns of a matrix
constexpr uint64_t kMaxK = uint64_t{1} << 21;       // of a product: 256 rows of codes, or of x, within 31 bits of bytes
constexpr uint64_t kMaxRows = 0x7FFFFFFFu;
constexpr uint64_t kMaxStride = uint64_t{1} << 32;
constexpr uint64_t kMaxValues = uint64_t{1} << 40;  // values of one matrix
constexpr uint64_t kMaxExtent = uint64_t{1} << 48;  // rows times stride
constexpr uint32_t kBlock = 32;                     // values that share a scale
constexpr uint32_t kNanScale = 255;

// ---- Quantisation ----------------------------------------------------------
// Four lanes take one block of 32 values, 8 values (16 bytes) each; the
// block's maximum goes round the four by two DPP exchanges.  An item is a
// block; items are numbered row by row, so that rows of any width fill the
// lanes.  Bound by HBM: 2 bytes read and 17/32 written for a value, and the
// other way round in the expansion: 4096 x 4096 in 9.8 and 9.3 us, 4.3 and 4.6
// TB/s (a large copy reaches 4.7); 9001 x 1387, rows that start at any even
// address, 9.0 and 8.1 us, where loads of one value at a time took 15.6 and 19.8.

constexpr uint32_t kQuantThreads = 256;
constexpr uint32_t kQuantItems = kQuantThreads / 4;  // blocks per workgroup and step

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    const uint32_t a = __builtin_amdgcn_update_dpp(0u, v, 0xB1, 0xF, 0xF, true);  // lanes 1 0 3 2
    v = v > a ? v : a;
    const uint32_t b = __builtin_amdgcn_update_dpp(0u, v, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
    return v > b ? v : b;
}

// 16 bytes of a row that may start at any even address: the hardware loads and
// stores them as they lie, without the compiler having to take them apart.
struct __attribute__((packed, aligned(2))) Piece {
    uint32_t w[4];
};

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
        if (col + 8 <= cols) {
            const Piece t = *reinterpret_cast<const Piece *>(src);
            w[0] = t.w[0], w[1] = t.w[1], w[2] = t.w[2], w[3] = t.w[3];
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
// takes the scale as a 32-bit float of which it reads the exponent.  Under an
// exponent of 255 every code gives NaN, that of zero too, which is what the
// product needs of a block with s = 255; the expansion writes one NaN for all.
template <int kByte>
__device__ __forceinline__ uint32_t expand2(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, kByte));
}

__device__ __forceinline__ v4u expand8(uint32_t codes, float scale) {
    return v4u{expand2<0>(codes, scale), expand2<1>(codes, scale), expand2<2>(codes, scale), expand2<3>(codes, scale)};
}

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
        if (col + 8 <= cols) {
            *reinterpret_cast<Piece *>(dst) = Piece{o.x, o.y, o.z, o.w};
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
    uint32_t m, n, k, blocks;  // blocks of 32 along k
    uint32_t y_wide;        // rows of y start at multiples of 16 bytes
    // tile form
    uint32_t tiles_m, tiles_n;
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    bf2 v;
    v.x = static_cast<__bf16>(a);
    v.y = static_cast<__bf16>(b);
    return __builtin_bit_cast(uint32_t, v);
}

typedef __attribute__((address_space(3))) void *LdsPtr;

// Waits for this wave's loads, those into LDS among them: a barrier alone does
// not (vmcnt 0; the other counters as they are).
__device__ __forceinline__ void arrived() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// Eight values of a row of k values, from column col on, zeros past its end.
__device__ __forceinline__ v4u piece_of(const uint16_t *row, uint32_t col, uint32_t k) {
    uint32_t w[4] = {0, 0, 0, 0};
    if (col + 8 <= k) {
        const Piece t = *reinterpret_cast<const Piece *>(row + col);
        w[0] = t.w[0], w[1] = t.w[1], w[2] = t.w[2], w[3] = t.w[3];
    } else if (col < k) {
#pragma unroll
        for (uint32_t i = 0; i < 7; ++i) {
            const uint32_t v = row[min(col + i, k - 1)];  // no branch for each value
            w[i / 2] |= (col + i < k ? v : 0u) << (16 * (i & 1));
        }
    }
    return v4u{w[0], w[1], w[2], w[3]};
}

// Token form, for few rows: a workgroup takes 16 kRows rows of w by kX of x, its
// waves share k between them and add their sums in LDS.  A lane reads 16 bytes
// of codes at a time, which is one block of one row: lane l has row l % 16 and
// block 4 s + l / 16 of step s.  The matrix instruction's k index is ours to
// choose, as long as both operands agree: its i-th instruction of a step takes
// codes 8 i .. 8 i + 7 of every lane's block, so nothing moves between lanes and
// one scale serves all of a lane's codes.
// Bound by HBM for the largest (1 x 128256 x 4096: 279 MB in 48 us, 5.8 TB/s), by
// a kernel's own start and end for the smallest (1 x 4096 x 4096: 4 us), and by
// the path of vector loads as soon as those are not few and wide.  So x comes
// in rows of 256 bytes a step by loads into the wave's own part of LDS, one
// instruction for 4 rows (piece c of row i lies at c ^ (i % 16), as in the tile
// form), and the scales of four steps in one load of 16 bytes.  With x read
// from memory in the order of the matrix instruction, four loads a step, and a
// byte of scales for each block, 1 x 128256 x 4096 took 88 us and 16 x 4096 x
// 14336 21 where it is 10.6 now.
//
// How it reads: kReadWide as above, for k in multiples of 512; kReadNarrow with
// a byte of scales for each block; kReadAny also takes rows of x that start
// anywhere and end inside a block, through registers.
enum TokenReads : int { kReadWide, kReadNarrow, kReadAny };

constexpr int kTokenWaves = 8;

template <int kX, int kRows, int kAhead, int kReads>
__global__ void __launch_bounds__(64 * kTokenWaves)
token_kernel(MulParams p) {
    constexpr bool kWide = kReads == kReadWide;
    constexpr int kM = kX < 16 ? 1 : kX / 16;        // tiles of x
    constexpr uint32_t kGroup = kWide ? 4 : kAhead;  // steps that a wave takes together: those whose scales are one load
    constexpr uint32_t kStepBytes = kX * 256, kWaveBytes = kAhead * kStepBytes;
    constexpr uint32_t kSumBytes = kM * kRows * 1024;  // of a wave
    __shared__ __attribute__((aligned(1024))) uint8_t s_x[kTokenWaves * (kWaveBytes > kSumBytes ? kWaveBytes : kSumBytes)];
    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t n0 = blockIdx.x * 16 * kRows, m0 = blockIdx.y * kX;
    const uint32_t rows_n = min(16u * kRows, p.n - n0), rows_m = min(uint32_t{kX}, p.m - m0);
    const Rsrc wr = rsrc(p.codes + uint64_t{n0} * p.blocks * 16, rows_n * p.blocks * 16);
    const Rsrc sr = rsrc(p.scales + uint64_t{n0} * p.blocks, rows_n * p.blocks);
    const uint32_t row_bytes = static_cast<uint32_t>(p.x_stride) * 2, k_bytes = p.blocks * kBlock * 2;
    const uint16_t *x0 = p.x + uint64_t{m0} * p.x_stride;
    const Rsrc xr = rsrc(x0, (rows_m - 1) * row_bytes + k_bytes);
    uint8_t *mine = s_x + wave * kWaveBytes;
    f4 acc[kM][kRows] = {};
    for (uint32_t g0 = wave * kGroup * 4; g0 < p.blocks; g0 += kTokenWaves * kGroup * 4) {
        uint32_t sc[kRows][kGroup];  // byte i of word a: the scale of block i of the group's step a in row r
        if (kWide) {
#pragma unroll
            for (uint32_t t = 0; t < kRows; ++t) {
                const v4u v = __builtin_amdgcn_raw_buffer_load_b128(sr, (r + 16 * t) * p.blocks + g0, 0, 0);
                sc[t][0] = v.x, sc[t][1] = v.y, sc[t][2] = v.z, sc[t][3] = v.w;
            }
        }
#pragma unroll
        for (uint32_t b0 = 0; b0 < kGroup; b0 += kAhead) {
            __builtin_amdgcn_s_waitcnt(0xC07F);  // what was read from LDS before has arrived (lgkmcnt 0)
            v4u c[kAhead][kRows], xs[kAhead][kX / 4];
#pragma unroll
            for (uint32_t a = 0; a < kAhead; ++a) {
                const uint32_t block0 = g0 + 4 * (b0 + a);  // past the end at most in the last group
                const uint32_t k0 = min(block0, p.blocks) * kBlock * 2;
#pragma unroll
                for (uint32_t j = 0; j < kX / 4; ++j) {
                    const uint32_t row = 4 * j + q, piece = (r ^ (row & 15u)) * 16;
                    if (kReads == kReadAny)
                        xs[a][j] = row < rows_m ? piece_of(x0 + row * p.x_stride, (k0 + piece) / 2, p.k) : v4u{0, 0, 0, 0};
                    else
                        __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (LdsPtr)(mine + a * kStepBytes + j * 1024), 16,
                                                                 k0 + piece < k_bytes ? row * row_bytes + piece : kOff,
                                                                 __builtin_amdgcn_readfirstlane(k0), 0, 0);
                }
                const uint32_t at = block0 + q < p.blocks ? r * p.blocks + block0 + q : kOff / 16;
#pragma unroll
                for (uint32_t t = 0; t < kRows; ++t) {
                    c[a][t] = __builtin_amdgcn_raw_buffer_load_b128(wr, (at + 16 * t * p.blocks) * 16, 0, 0);
                    if (!kWide)
                        sc[t][b0 + a] = (__builtin_amdgcn_raw_buffer_load_b8(sr, at + 16 * t * p.blocks, 0, 0) & 255u)
                                        << (8 * q);
                }
            }
            if (kReads == kReadAny) {
#pragma unroll
                for (uint32_t a = 0; a < kAhead; ++a)
#pragma unroll
                    for (uint32_t j = 0; j < kX / 4; ++j)
                        *reinterpret_cast<v4u *>(mine + a * kStepBytes + j * 1024 + lane * 16) = xs[a][j];
            } else {
                arrived();
            }
#pragma unroll
            for (uint32_t a = 0; a < kAhead; ++a) {
                float scale[kRows];
#pragma unroll
                for (uint32_t t = 0; t < kRows; ++t)
                    scale[t] = __builtin_bit_cast(float, (sc[t][b0 + a] >> (8 * q) & 255u) << 23);
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) {
                    bf8 xf[kM];
#pragma unroll
                    for (uint32_t u = 0; u < kM; ++u) {
                        const uint32_t row = kX < 16 ? r % kX : 16 * u + r;  // rows past kX repeat: columns not stored
                        xf[u] = *reinterpret_cast<const bf8 *>(mine + a * kStepBytes + row * 256 +
                                                               ((4 * q + i) ^ (row & 15u)) * 16);
                    }
#pragma unroll
                    for (uint32_t t = 0; t < kRows; ++t) {
                        const bf8 wf = __builtin_bit_cast(bf8, expand8(c[a][t][i], scale[t]));
#pragma unroll
                        for (uint32_t u = 0; u < kM; ++u)
                            acc[u][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[u], acc[u][t], 0, 0, 0);
                    }
                }
            }
        }
    }
    // acc: column lane % 16 (a row of x), rows 4 (lane / 16) + 0..3 (of w)
    __syncthreads();  // the sums go where x was
    float *sum = reinterpret_cast<float *>(s_x);
#pragma unroll
    for (uint32_t u = 0; u < kM; ++u)
#pragma unroll
        for (uint32_t t = 0; t < kRows; ++t)
            *reinterpret_cast<f4 *>(sum + ((wave * kM + u) * kRows + t) * 256 + r * 16 + 4 * q) = acc[u][t];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < kM * kRows * 256; i += 64 * kTokenWaves) {
        // neighbouring threads take neighbouring columns of a row
        const uint32_t col = i % (16 * kRows), row = i / (16 * kRows);
        const uint32_t at = ((row / 16) * kRows + col / 16) * 256 + row % 16 * 16 + col % 16;
        float v = 0;
#pragma unroll
        for (uint32_t k = 0; k < kTokenWaves; ++k) v += sum[k * kM * kRows * 256 + at];
        if (row < rows_m && col < rows_n)
            p.y[uint64_t{m0 + row} * p.y_stride + n0 + col] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
    }
}

// Tile form, for many rows: a workgroup computes a tile of 16 kTiles rows of x
// by 64 kCols rows of w, each wave of a group of four 16 kTiles by 16 kCols of
// it, in stages of 128 along k; two groups take the stages in turn and add their
// sums.  x goes to LDS by loads that write there directly, two stages, the next
// one loading while one is computed.  The codes go from memory to the registers
// of the waves that use them and are expanded there: a lane's 16 bytes are one
// block of 32, k as in the token form.  A row of x in LDS is 16 pieces of 16
// bytes; piece c of row i lies at c ^ (i % 16), so that the 16 rows a read
// touches use all banks once.  Row m of a wave's t-th tile of w is row
// 4 kCols (m / 4) + 4 t + m % 4 of its 16 kCols, which leaves a lane with
// 4 kCols neighbouring columns of y in the end.
// Scales come with kWide, for k in multiples of 512, for four stages at a time
// and through LDS like x; else by a byte for each block (8192 x 8192 x 8192: 744
// us against 805; it costs more where tiles are many and k is long: 64 x 256
// tiles of 1792 x 4096 take 199 us for k of 14,336 and 198 for 11,008).
// Bound by the matrix unit, held back by the loads of a stage: 8192 x 8192 x 8192
// in 744 us, 1.48 PFLOP/s (a large BF16 product of the vendor's library reaches
// 1.39 on the same card), 2048 x 14336 x 4096 in 186, 1.30; expanding the codes
// costs nothing beside the matrix instructions.  Two workgroups of four waves
// on a compute unit hide one another's barriers: one of eight waves and 256
// rows was no faster (204 us against 197 for 2048 x 14336 x 4096 at the time).
constexpr uint32_t kStageK = 128;
constexpr uint32_t kStageBlocks = kStageK / kBlock;
constexpr uint32_t kRowBytes = kStageK * 2;

constexpr uint32_t kTileWaves = 4;
constexpr uint32_t kBand = 8;

template <int kTiles, int kCols, int kGroups, bool kWide>
__global__ void __launch_bounds__(64 * kTileWaves * kGroups) __attribute__((amdgpu_waves_per_eu(2)))
tile_kernel(MulParams p) {
    constexpr uint32_t kRowsM = 16 * kTiles, kWaveN = 16 * kCols, kRowsN = kWaveN * kTileWaves;
    constexpr int kLoads = kRowsM / 4 / kTileWaves;  // a wave's loads of a stage: 4 rows each, 16 rows from one another
    constexpr uint32_t kGroupBytes = 2 * kRowsM * kRowBytes;  // two stages; as many bytes as a group's sums
    __shared__ __attribute__((aligned(1024))) uint8_t s_all[kGroups * kGroupBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t s_scale[kWide ? kGroups * kTileWaves * 2 * 1024 : 16];

    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, q = lane >> 4;
    const uint32_t group = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / kTileWaves;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % kTileWaves;
    uint8_t *s_x = s_all + group * kGroupBytes;
    // workgroups go round the 8 XCDs; each XCD takes a run of neighbouring
    // tiles, in bands of 8 tiles along m, so that its L2 holds what the tiles of
    // the moment share (8192 x 8192 x 8192: 854 us with all of m in a band, 805 in
    // bands of 8 at the time)
    const uint32_t tiles = p.tiles_m * p.tiles_n, per = tiles / 8, more = tiles % 8, xcd = blockIdx.x % 8;
    const uint32_t t = xcd * per + min(xcd, more) + blockIdx.x / 8;
    const uint32_t band = t / (kBand * p.tiles_n), in_band = t - band * kBand * p.tiles_n;
    const uint32_t width = min(kBand, p.tiles_m - band * kBand);
    const uint32_t m0 = (band * kBand + in_band % width) * kRowsM, n0 = in_band / width * kRowsN;

    const uint32_t stages = (p.blocks + kStageBlocks - 1) / kStageBlocks;

    // Rows past m and n, and blocks past k, lie past their resource and read as
    // zero; the scalar offsets stay within it.
    // x: lane l of a load has row l / 16 of four, of it piece l % 16 in LDS
    const uint32_t row_bytes = static_cast<uint32_t>(p.x_stride) * 2, k_bytes = p.blocks * kBlock * 2;
    const Rsrc xr = rsrc(p.x + uint64_t{m0} * p.x_stride, (min(kRowsM, p.m - m0) - 1) * row_bytes + k_bytes);
    const uint32_t x_piece = (r ^ ((4 * wave + q) & 15u)) * 16;
    const uint32_t x_off = (4 * wave + q) * row_bytes + x_piece;
    // w: the lane's row of the wave's first tile
    const uint32_t rows_n = min(kRowsN, p.n - n0);
    const Rsrc wr = rsrc(p.codes + uint64_t{n0} * p.blocks * 16, rows_n * p.blocks * 16);
    const Rsrc sr = rsrc(p.scales + uint64_t{n0} * p.blocks, rows_n * p.blocks);
    const uint32_t w_off = (kWaveN * wave + 4 * kCols * (r / 4) + r % 4) * p.blocks + q;

    auto load_x = [&](uint32_t stage, uint8_t *to) {
        const uint32_t k0 = __builtin_amdgcn_readfirstlane(stage * kRowBytes);
        const uint32_t off = k0 + x_piece < k_bytes ? x_off : kOff;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (LdsPtr)(to + (i * kTileWaves + wave) * 1024), 16,
                                                     off + 4 * kTileWaves * i * row_bytes, k0, 0, 0);
    };
    // scales of the wave's rows: 16 bytes of a row, four stages', in one load (of 64
    // rows: with kCols of 2 the other half are not its own) into the wave's part of
    // LDS, two parts in turn
    uint8_t *scale_part = s_scale + (group * kTileWaves + wave) * 2048;
    auto load_scales = [&](uint32_t four) {
        const uint32_t row = kWaveN * wave + lane;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(sr, (LdsPtr)(scale_part + (four & 1) * 1024), 16, row * p.blocks,
                                                 __builtin_amdgcn_readfirstlane(four * 16), 0, 0);
    };
    struct W {
        v4u code[kCols];
        uint32_t scale[kCols];
    };
    auto load_w = [&](uint32_t stage, W &w) {
        const uint32_t at = __builtin_amdgcn_readfirstlane(stage * kStageBlocks);
        const bool in = at + q < p.blocks;
        const uint32_t code_off = in ? w_off * 16 : kOff, scale_off = in ? w_off : kOff;
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
            w.code[i] = __builtin_amdgcn_raw_buffer_load_b128(wr, code_off + 4 * i * p.blocks * 16, at * 16, 0);
            if (!kWide) w.scale[i] = __builtin_amdgcn_raw_buffer_load_b8(sr, scale_off + 4 * i * p.blocks, at, 0);
        }
    };
    auto read_scales = [&](uint32_t stage, W &w) {
        const uint8_t *at = scale_part + (stage / 4 & 1) * 1024 + (4 * kCols * (r / 4) + r % 4) * 16 + stage % 4 * 4 + q;
#pragma unroll
        for (int i = 0; i < kCols; ++i) w.scale[i] = at[4 * i * 16];
    };

    // Stage: 4 steps of 32 along k, in each 4 kTiles matrix instructions.  A
    // piece of x is read for the next step as soon as this step is done with
    // the registers it goes to, and the next step's codes are expanded beside;
    // the order is given to the compiler in groups (left to itself it read just
    // before use: 2048 x 14336 x 4096 239 us against 212, in tiles of 256 rows).
    f4 acc[kTiles][kCols] = {};
    auto expand = [&](const W &w, int j, bf8 (&to)[kCols]) {
#pragma unroll
        for (int i = 0; i < kCols; ++i)
            to[i] = __builtin_bit_cast(bf8, expand8(w.code[i][j], __builtin_bit_cast(float, (w.scale[i] & 255u) << 23)));
    };
    auto compute = [&](const uint8_t *x, const W &w) {
        const uint8_t *row = x + r * kRowBytes;
        bf8 xf[kTiles], wf[2][kCols];
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
            xf[m] = *reinterpret_cast<const bf8 *>(row + m * 16 * kRowBytes + ((4 * q) ^ r) * 16);
        expand(w, 0, wf[0]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t piece = ((4 * q + j + 1) ^ r) * 16;
            if (j < 3) expand(w, j + 1, wf[(j + 1) & 1]);
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
#pragma unroll
                for (int i = 0; i < kCols; ++i)
                    acc[m][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[j & 1][i], xf[m], acc[m][i], 0, 0, 0);
                if (j < 3) xf[m] = *reinterpret_cast<const bf8 *>(row + m * 16 * kRowBytes + piece);
            }
            if (j < 3) {
#pragma unroll
                for (int m = 0; m < kTiles; ++m) {
                    __builtin_amdgcn_sched_group_barrier(0x008, kCols / 2, 0);         // matrix instructions
                    __builtin_amdgcn_sched_group_barrier(0x002, 4 * kCols / kTiles, 0);  // expansion
                    __builtin_amdgcn_sched_group_barrier(0x008, kCols / 2, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                 // LDS read
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    W w, next;
    if (group < stages) {
        load_x(group, s_x);
        load_w(group, w);
        if (kWide) load_scales(group / 4);
    }
    uint32_t flip = 0;
    for (uint32_t s0 = 0; s0 < stages; s0 += kGroups) {  // the same count for all waves, which meet in it
        const uint32_t s = s0 + group;
        arrived();
        __syncthreads();  // stage s is there, the one before is read
        const uint32_t other = flip ^ (kRowsM * kRowBytes);
        if (s + kGroups < stages) {
            load_x(s + kGroups, s_x + other);
            load_w(s + kGroups, next);
            if (kWide && (s + kGroups) / 4 != s / 4) load_scales((s + kGroups) / 4);
        }
        if (s < stages) {
            if (kWide) read_scales(s, w);
            compute(s_x + flip, w);
        }
        w = next;
        flip = other;
    }
    if (kGroups > 1) {  // the other groups' sums through LDS to the first
        static_assert((kGroups - 1) * kRowsM * kRowsN * 4 <= kGroups * kGroupBytes, "the groups' sums fit");
        f4 *sum = reinterpret_cast<f4 *>(s_all) + (wave * 64 + lane);
        __syncthreads();
        if (group > 0) {
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int i = 0; i < kCols; ++i) sum[(((group - 1) * kTiles + m) * kCols + i) * 64 * kTileWaves] = acc[m][i];
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g = 0; g < kGroups - 1; ++g)
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int i = 0; i < kCols; ++i) acc[m][i] += sum[((g * kTiles + m) * kCols + i) * 64 * kTileWaves];
    }

    // a lane: 4 kCols columns of the wave's 16 kCols, row r of each tile
    const uint32_t col = n0 + kWaveN * wave + 4 * kCols * q;
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
        const uint32_t row = m0 + 16 * m + r;
        if (row >= p.m || col >= p.n) continue;
        uint16_t *to = p.y + uint64_t{row} * p.y_stride + col;
        uint32_t o[2 * kCols];
#pragma unroll
        for (int i = 0; i < 2 * kCols; ++i) o[i] = pack2(acc[m][i / 2][2 * (i & 1)], acc[m][i / 2][2 * (i & 1) + 1]);
        if (p.y_wide && col + 4 * kCols <= p.n) {
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i)
                *reinterpret_cast<v4u *>(to + 8 * i) = v4u{o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]};
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 4 * kCols; ++i)
                if (col + i < p.n) to[i] = static_cast<uint16_t>(o[i / 2] >> (16 * (i & 1)));
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
           (rows == 0 || stride <= kMaxExtent / rows);
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
    return launched(launch(quantize_kernel, dim3(quant_grid(items)), kQuantThreads,
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
    return launched(launch(dequantize_kernel, dim3(quant_grid(items)),
                           kQuantThreads, static_cast<hipStream_t>(hip_stream), codes, scales,
                           static_cast<uint32_t>(cols), blocks, items, out, out_stride));
}

// The form of a product.  A workgroup of the token form takes a piece of 4, 16,
// 32 or 64 rows of x by 16, 32 or 64 of w, one of the tile form 64 rows of x by 128 or
// 256 of w or 128 by 256.
//  - Up to 32 rows, and as long as 64 x 64 pieces make no more than one for each of
//    256 compute units, the token form, whose waves share k, is the faster one: 256 x
//    4096 x 4096 (256 pieces) 17.9 us against 24.5 for the best tiles, 320 (320) 32.4
//    against 24.9, 96 x 14336 x 4096 (448) 33.4 against 26.2.  Where k is at most 1,024
//    a wave has little to do, and half as many pieces are the limit: 256 x 4096 x 512
//    (256) 7.8 against 5.8, 128 x 4096 x 512 (128) 5.4 against 5.6.
//  - In the token form the largest piece that leaves 160 workgroups (256 of
//    16 rows): 64 x 4096 x 4096 8.2 us by 32 x 32 (256 workgroups), 10.8 by 64 x 32 (128)
//    and 15.8 by 64 x 64 (64); 16 x 14336 x 4096 9.5 by 16 x 32 (448), 10.1 by 16 x 64 (224),
//    11.7 by 16 x 16.
//  - Tiles of 64 x 128 up to three for each compute unit, four of which fit it at a
//    time: 1536 x 4096 x 4096 (768 tiles) 49.3 us against 51.2 for 64 x 256, 384 x 14336 x
//    4096 (672) 46.9 against 52.1, 512 x 14336 x 4096 (896) 63.3 against 54.8.
//  - Larger ones of 64 or 128 rows, by the tiles of 128 rows that there would be (us with 64
//    and with 128; k of 2,080 and 11,008 is read with a byte of scales for each block):
//      up to 256, one for a compute unit, where 128 has two groups of waves: 1792 x 4096 (224)
//      with k of 1,024, 4,096, 14,336: 24.5 and 25.9, 61.5 and 60.9, 199 and 193, of 1,056,
//      2,080, 11,008: 27.5 and 27.8, 40.7 and 39.5, 198 and 148.  832 x 8192 the same, but for
//      k of 4,096: 59.3 and 61.7;
//      up to 384: 2304 x 4096 (288) with k of 1,024, 4,096, 14,336: 30.5 and 34.2, 87.4 and
//      96.3, 283 and 271, of 1,056, 2,080, 11,008: 33.5 and 37.5, 53.5 and 59.9, 286 and 260;
//      1536 x 8192 (384) with k of 14,336: 310 and 320, of 11,008 298 and 264;
//      past 384: 1664 x 8192 (416) with k of 1,024, 4,096, 14,336: 38.3 and 36.2, 118 and 102,
//      381 and 316.  Past 512 a last round that is not full favours 64 by up to a tenth (576,
//      2304 x 8192 x 4096: 139 and 152), a full one 128 (1,024: 231 and 218; 1,792: 405 and 367).
//  - Two groups of waves in a tile, which take stages in turn, up to 256 tiles, one for a
//    compute unit: 512 x 4096 x 4096 in 64 x 128 27.6 us against 32.3, 1792 x 4096 x 4096 in
//    128 x 256 60.9 against 69.2; with more tiles other workgroups are there to fill the
//    waits (768 x 4096 x 4096, 384 tiles of 64 x 128: 37.0 against 34.7).
struct Form {
    bool token;
    uint32_t x, rows;  // of x and of w in a piece or tile; token form: tiles of 16 rows of w
};

uint64_t pieces(uint64_t m, uint64_t x, uint64_t n, uint64_t w) { return ((m + x - 1) / x) * ((n + w - 1) / w); }

// Whether tiles of 128 rows, of which there would be this many, take less time than those of 64.
bool large_tiles(uint64_t tiles, uint64_t k) {
    const bool narrow = k % 512 != 0;  // scales by the byte
    if (tiles <= 256) return k > (narrow ? 1536 : 4096);
    return tiles > 384 || (narrow && k > 8192);
}

Form form_of(uint64_t m, uint64_t n, uint64_t k) {
    if (m <= 4) return {true, 4, 1};
    if (m > 32 && pieces(m, 64, n, 64) > (k <= 1024 ? 128 : 256)) {
        if (pieces(m, 64, n, 128) <= 768) return {false, 64, 128};
        return {false, large_tiles(pieces(m, 128, n, 256), k) ? 128u : 64u, 256};
    }
    if (m > 32)
        for (uint32_t rows : {4u, 2u})
            if (pieces(m, 64, n, 16 * rows) >= 160) return {true, 64, rows};
    if (m > 16)
        for (uint32_t rows : {4u, 2u})
            if (pieces(m, 32, n, 16 * rows) >= 160) return {true, 32, rows};
    for (uint32_t rows : {4u, 2u})
        if (pieces(m, 16, n, 16 * rows) >= 256) return {true, 16, rows};
    return {true, 16, 1};
}

// Whether a product's work items fit a launch, which holds fewer than 2^32 in a
// dimension; the token form's other dimension has at most 1,024 workgroups.
bool launchable(const Form &f, uint64_t m, uint64_t n) {
    const uint64_t groups = f.token ? pieces(1, 1, n, 16 * f.rows) : pieces(m, f.x, n, f.rows);
    return groups * 64 * (f.token ? kTokenWaves : kTileWaves) < uint64_t{1} << 32;
}

template <int kX, int kRows, int kAhead>
hipError_t launch_token(int reads, hipStream_t st, const MulParams &p) {
    const dim3 grid((p.n + 16 * kRows - 1) / (16 * kRows), (p.m + kX - 1) / kX);
    return launch(reads == kReadWide     ? token_kernel<kX, kRows, kAhead, kReadWide>
                  : reads == kReadNarrow ? token_kernel<kX, kRows, kAhead, kReadNarrow>
                                         : token_kernel<kX, kRows, kAhead, kReadAny>,
                  grid, 64 * kTokenWaves, st, p);
}

template <int kTiles, int kCols, int kGroups>
hipError_t launch_tile(bool wide, dim3 grid, hipStream_t st, const MulParams &p) {
    return launch(wide ? tile_kernel<kTiles, kCols, kGroups, true> : tile_kernel<kTiles, kCols, kGroups, false>, grid,
                  64 * kTileWaves * kGroups, st, p);
}

// Rows of x are read 16 bytes and whole blocks at a time, with byte offsets of
// 31 bits in a tile.  The token form has another way for those that cannot be
// (kReadAny); for the tile form they are copied into the workspace first.
constexpr uint64_t kMaxRead = uint64_t{1} << 21;  // stride of x for 256 rows in 2^30 bytes

uint64_t copy_bytes(uint64_t m, uint64_t n, uint64_t k, bool x_readable) {
    if ((x_readable && k % kBlock == 0) || m == 0 || n == 0 || form_of(m, n, k).token) return 0;
    return (m * ((k + kBlock - 1) / kBlock) * kBlock * 2 + 15) / 16 * 16;
}

df11_status matmul(const uint16_t *x, uint64_t m, uint64_t k, uint64_t x_stride, const uint8_t *codes,
                   const uint8_t *scales, uint64_t n, uint16_t *y, uint64_t y_stride, void *workspace,
                   uint64_t workspace_bytes, void *hip_stream) {
    if (m > kMaxRows || n > kMaxRows || k > kMaxK || x_stride > kMaxStride || x_stride < k || y_stride < n ||
        y_stride > kMaxStride || m * std::max(x_stride, y_stride) > kMaxExtent)
        return DF11_E_INVALID_ARG;
    if (m == 0 || n == 0) return DF11_OK;
    if (!y || (k && (!x || !codes || !scales)) || !aligned16(codes) || (reinterpret_cast<uintptr_t>(x) & 1u) ||
        (reinterpret_cast<uintptr_t>(y) & 1u) || !aligned16(workspace))
        return DF11_E_INVALID_ARG;
    const bool readable = aligned16(x) && x_stride % 8 == 0 && x_stride <= kMaxRead;
    const Form f = form_of(m, n, k);
    if (!launchable(f, m, n)) return DF11_E_INVALID_ARG;
    const uint64_t copy = copy_bytes(m, n, k, readable);
    if (workspace_bytes < copy) return DF11_E_BUFFER_TOO_SMALL;
    if (copy && !workspace) return DF11_E_INVALID_ARG;
    const uint64_t tiles = f.token ? 0 : pieces(m, f.x, n, f.rows);
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    MulParams p = {};
    p.x = x;
    p.codes = codes;
    p.scales = scales;
    p.y = y;
    p.x_stride = x_stride;
    p.y_stride = y_stride;
    p.m = static_cast<uint32_t>(m);
    p.n = static_cast<uint32_t>(n);
    p.k = static_cast<uint32_t>(k);
    p.blocks = static_cast<uint32_t>((k + kBlock - 1) / kBlock);
    p.y_wide = aligned16(y) && y_stride % 8 == 0;
    hipError_t err = hipSuccess;
    if (copy) {
        const uint32_t width = p.blocks * kBlock;
        const uint64_t lanes = m * (width / 8);
        err = launch(pack_rows_kernel, dim3(static_cast<uint32_t>(std::min<uint64_t>((lanes + 255) / 256, 8192))), 256,
                     st, x, x_stride, static_cast<uint32_t>(k), width, m, static_cast<uint16_t *>(workspace));
        if (err != hipSuccess) return launched(err);
        p.x = static_cast<const uint16_t *>(workspace);
        p.x_stride = width;
    }
    const bool wide = p.blocks % 16 == 0 && aligned16(scales);
    if (f.token) {
        // kReadWide gives a wave 512 of k at a time: below 2,048 that leaves more
        // than half of the waves idle (512 x 4096 x 1024 in pieces 18.7 us against 16.5; at
        // 2,048 16 x 14336 takes 6.1 against 7.5)
        const int reads = !readable || k % kBlock != 0 ? kReadAny : wide && p.blocks >= 64 ? kReadWide : kReadNarrow;
        switch (f.x + f.rows) {
            case 4 + 1: return launched(launch_token<4, 1, 4>(reads, st, p));
            case 16 + 1: return launched(launch_token<16, 1, 2>(reads, st, p));
            case 16 + 2: return launched(launch_token<16, 2, 2>(reads, st, p));
            case 16 + 4: return launched(launch_token<16, 4, 2>(reads, st, p));
            case 32 + 2: return launched(launch_token<32, 2, 2>(reads, st, p));
            case 32 + 4: return launched(launch_token<32, 4, 2>(reads, st, p));
            case 64 + 2: return launched(launch_token<64, 2, 1>(reads, st, p));
            default: return launched(launch_token<64, 4, 1>(reads, st, p));
        }
    }
    p.tiles_m = static_cast<uint32_t>((m + f.x - 1) / f.x);
    p.tiles_n = static_cast<uint32_t>((n + f.rows - 1) / f.rows);
    const dim3 grid(static_cast<uint32_t>(tiles));
    const bool two = tiles <= 256;
    if (f.rows == 128) return launched(two ? launch_tile<4, 2, 2>(wide, grid, st, p) : launch_tile<4, 2, 1>(wide, grid, st, p));
    if (f.x == 64) return launched(launch_tile<4, 4, 1>(wide, grid, st, p));  // always more than 256 tiles
    return launched(two ? launch_tile<8, 4, 2>(wide, grid, st, p) : launch_tile<8, 4, 1>(wide, grid, st, p));
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
    if (m > kMaxRows || n > kMaxRows || k > kMaxK || !launchable(form_of(m, n, k), m, n)) return 0;  // refused by the product
    return copy_bytes(m, n, k, x_aligned != 0);
}

extern "C" df11_status df11_mx4_matmul(const uint16_t *x, uint64_t m, uint64_t k, uint64_t x_stride,
                                       const uint8_t *codes, const uint8_t *scales, uint64_t n, uint16_t *y,
                                       uint64_t y_stride, void *workspace, uint64_t workspace_bytes,
                                       void *hip_stream) {
    return df11i::guarded([&] {
        return matmul(x, m, k, x_stride, codes, scales, n, y, y_stride, workspace, workspace_bytes, hip_stream);
    });
}
