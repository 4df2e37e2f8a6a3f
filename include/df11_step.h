/*
 * df11_step.h -- the part of libdf11 that a token step calls besides the
 * block decode of df11.h, on an AMD Instinct MI355X (gfx950): two more stores
 * of what a step reads, each with the operator that reads it without
 * expanding it in memory.
 *
 *  - Weights in microscaled 4-bit floating point ("MX4"): 32 consecutive
 *    values of a row share one power of two, each value is a 4-bit float
 *    (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6).
 *    17/32 byte for a weight; lossy, unlike DF11.
 *  - Keys and values in a paged cache: pages of a fixed number of positions,
 *    found through a table for each sequence; BF16, or E4M3 (8-bit float with
 *    4 exponent bits) with one scale for each head.
 *
 * Every call is ordered on `hip_stream` (a hipStream_t; NULL = the null
 * stream), launches on the current device, neither synchronizes nor
 * allocates, and can be captured into a graph.  Arguments are checked on the
 * host before anything is launched.  Status codes are those of df11.h.
 * Strides count elements, not bytes.
 */
#ifndef DF11_STEP_H
#define DF11_STEP_H

#include "df11.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- 4-bit weights ------------------------------------------------------
 * A matrix of rows x cols values is stored as
 *   codes   rows x 16 * B bytes, B = ceil(cols / 32): byte j of a row holds
 *           the code of column 2j in its low half and of 2j + 1 in its high
 *           half (bit 3 sign, bits 2..1 exponent, bit 0 mantissa); columns
 *           past cols hold code 0
 *   scales  rows x B bytes: byte s scales block b (columns 32b..32b+31) by
 *           2^(s - 127); s = 255 says that the block holds an infinity or a
 *           NaN, and all of its values read as NaN. */

/* Quantises x (BF16 bit patterns, row_stride >= cols).  For a block with
 * largest magnitude a: scale 2^e, e = floor(log2 a) - 2 held to [-127, 127]
 * (-127 for a block of zeros); each code is the nearest grid value of x 2^-e,
 * of two as near the even code, magnitudes over 6 become 6, the sign is kept.
 * A block with an infinity or a NaN gets s = 255 and codes 0.  codes and
 * scales: device memory, codes 16-byte aligned.  rows = 0 is a no-op.
 * Errors: DF11_E_INVALID_ARG (null or misaligned pointers, cols = 0, a
 * stride below cols, more than 2^40 values or 2^24 columns), DF11_E_HIP. */
df11_status df11_mx4_quantize(const uint16_t *x, uint64_t rows, uint64_t cols, uint64_t row_stride,
                              uint8_t *codes, uint8_t *scales, void *hip_stream);

/* out (BF16, out_stride >= cols) := the values that codes and scales stand
 * for.  Exact: the smallest, 2^-128, is a BF16 denormal.  Those of 2^128 and
 * more (s of 253 and 254, which df11_mx4_quantize does not write) become
 * infinities, in the product too.  Errors as above. */
df11_status df11_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, uint64_t rows, uint64_t cols,
                                uint16_t *out, uint64_t out_stride, void *hip_stream);

/* y[i, j] = sum over k of x[i, k] w[j, k], i < m, j < n: activations x (BF16,
 * m x k) times 4-bit weights w (n x k as above, codes 16-byte aligned), the
 * products exact and summed in 32 bits, one rounding to BF16 (nearest even).
 * workspace: df11_mx4_matmul_workspace_bytes bytes of device memory, 16-byte
 * aligned (NULL when that is 0); its contents need not be kept or cleared.
 * m = 0 or n = 0 is a no-op; k = 0 gives zeros.  The result does not depend
 * on what runs beside it: every sum has a fixed order.  y must not overlap
 * the inputs.  Errors: DF11_E_INVALID_ARG (null or misaligned pointers,
 * strides below k or n or over 2^32, m times a stride over 2^48, m or n over
 * 2^31 - 1, k over 2^21, more rows of w than a launch holds: 2^27 with up to 4
 * rows of x, 2^29 with up to 32, m n of 2^37 with more), DF11_E_BUFFER_TOO_SMALL
 * (workspace_bytes), DF11_E_HIP. */
df11_status df11_mx4_matmul(const uint16_t *x, uint64_t m, uint64_t k, uint64_t x_stride, const uint8_t *codes,
                            const uint8_t *scales, uint64_t n, uint16_t *y, uint64_t y_stride, void *workspace,
                            uint64_t workspace_bytes, void *hip_stream);

/* Bytes of workspace for a product: 0, but for many rows of x that cannot be
 * read 16 bytes at a time or with k no multiple of 32 (a packed copy of x).
 * x_aligned: whether x is 16-byte aligned with x_stride a multiple of 8 and at
 * most 2^21. */
uint64_t df11_mx4_matmul_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, int32_t x_aligned);

/* ---- Paged key-value cache ----------------------------------------------
 * K and V pages: n_pages pages of page_size positions for kv_heads heads of
 * head_dim values each, head_dim values next to each other, the rest by
 * strides: the row of position r of head h in page p starts at
 * pages + p * page_stride + h * head_stride + r * row_stride.  Rows start at
 * multiples of 16 bytes.  head_dim 64, 128 or 256; page_size a power of two
 * from 8 to 1024; kv_heads up to 65536; n_pages below 2^31; strides up to
 * 2^40, and n_pages, kv_heads and page_size times their strides below 2^48
 * together. */
#define DF11_CACHE_BF16 0u
#define DF11_CACHE_E4M3 1u

typedef struct df11_paged_cache {
    void *k_pages, *v_pages;
    uint64_t n_pages;
    uint64_t k_page_stride, k_head_stride, k_row_stride; /* elements */
    uint64_t v_page_stride, v_head_stride, v_row_stride;
    const float *k_scale, *v_scale; /* E4M3: device, kv_heads scales each; BF16: NULL */
    uint32_t kv_heads, head_dim, page_size;
    uint32_t dtype;                 /* DF11_CACHE_* */
} df11_paged_cache;

/* Writes the keys and values of `tokens` tokens into the cache.  k, v: BF16,
 * token t of head h at k + t * k_token_stride + h * k_head_stride.  slots:
 * device, one 64-bit number for each token, page * page_size + position in
 * the page; a slot below 0 or past the cache is skipped (padding).  E4M3: the
 * stored value is x / scale[h] rounded to nearest even, magnitudes over 448
 * (infinities too) become 448, NaN stays NaN.  Of two tokens with one slot each
 * 8 values are either's.  tokens = 0 is a no-op.  Errors: DF11_E_INVALID_ARG (null
 * or misaligned pointers, sizes past the limits above, 2^31 tokens or more,
 * strides over 2^40 or, times what they step over, 2^48 together),
 * DF11_E_UNSUPPORTED (head_dim, page_size or dtype), DF11_E_HIP. */
df11_status df11_paged_append(const df11_paged_cache *cache, const uint16_t *k, uint64_t k_token_stride,
                              uint64_t k_head_stride, const uint16_t *v, uint64_t v_token_stride,
                              uint64_t v_head_stride, const int64_t *slots, uint64_t tokens, void *hip_stream);

/* Attention of one new token for each of `batch` sequences over the cache.
 * q: BF16, head g of sequence b at q + b * q_batch_stride + g * q_head_stride;
 * q_heads a multiple of kv_heads, query heads g with g / (q_heads / kv_heads)
 * = h read cache head h.  Sequence b reads positions j in [starts[b],
 * lens[b]) (device, 32-bit; starts NULL = 0; both held to [0, table_width *
 * page_size]); position j lies in page page_table[b * table_stride + j /
 * page_size].  A table entry outside [0, n_pages) masks its positions.  With
 * s_j = scale * q . k_j:
 *   out[b, g, :] = sum_j exp(s_j) v_j / sum_j exp(s_j)   (BF16, contiguous,
 *                  16-byte aligned)
 *   lse[b, g]    = log sum_j exp(s_j)                    (32 bits; NULL = not wanted)
 * and where that sum is zero (no position is left, or only scores of
 * -infinity), zeros and -infinity.  What masked positions hold, NaN included,
 * does not matter.  An infinity in v_j gives infinities of its sign (and with
 * one of the other sign, NaN), if exp(s_j) is above 2^-126 of the largest:
 * below, a weight is zero in 32 bits, and zero times infinity NaN.  Scores,
 * maxima, sums and the weighted values are held in 32 bits (their sum before
 * the division, which values of 2^128 over the number of positions can take
 * past the largest number); the weights exp(s_j) enter the product as two BF16
 * parts (16 bits of mantissa).  The result does not depend on what runs
 * beside it.  workspace: df11_paged_attention_workspace_bytes bytes of device
 * memory, 16-byte aligned (NULL when that is 0), not kept between calls;
 * calls that run at the same time need one each.  batch = 0 is a no-op.
 * page_table, lens and starts must not be written to while the call runs.
 * Errors: DF11_E_INVALID_ARG (null or misaligned pointers; table_width 0, or
 * 2^31 positions or more in it; table_stride below table_width; strides as for
 * the append; more than 2^20 query heads; more than a launch holds: batch x
 * kv_heads x ceil(q_heads / kv_heads / 16), times the chunks of a sequence
 * where they are split, below 2^24, and there batch x q_heads too),
 * DF11_E_UNSUPPORTED (as above), DF11_E_BUFFER_TOO_SMALL (workspace_bytes),
 * DF11_E_HIP. */
df11_status df11_paged_attention(const df11_paged_cache *cache, const uint16_t *q, uint64_t batch, uint64_t q_heads,
                                 uint64_t q_batch_stride, uint64_t q_head_stride, const int32_t *page_table,
                                 uint64_t table_stride, uint64_t table_width, const int32_t *lens,
                                 const int32_t *starts, float scale, uint16_t *out, float *lse, void *workspace,
                                 uint64_t workspace_bytes, void *hip_stream);

/* Bytes of workspace for an attention call (0 where a sequence's positions
 * are not split). */
uint64_t df11_paged_attention_workspace_bytes(uint64_t batch, uint64_t q_heads, uint32_t kv_heads, uint32_t head_dim,
                                              uint32_t page_size, uint64_t table_width);

#ifdef __cplusplus
}
#endif

#endif /* DF11_STEP_H */
