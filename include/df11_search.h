/*
 * df11_search.h -- the part of libdf11 that decodes with more than one
 * candidate for each sequence, over the paged cache of df11_step.h, on an AMD
 * Instinct MI355X (gfx950):
 *
 *  - attention of a tree of drafted tokens (or of a chain of new ones, such as
 *    a chunk of a prompt) over the cache;
 *  - the cache's pages after the choice: an accepted path made contiguous
 *    (compact), rows of the page table reordered with their pages shared, taken
 *    and given back by counts that stay on the device (fork), the pages that a
 *    fork has to copy, or any others (copy);
 *  - the selection of a beam search, whose parents are those of a fork.
 *
 * Calls follow df11_step.h: ordered on `hip_stream`, on the current device,
 * without synchronizing or allocating, capturable into a graph, arguments
 * checked on the host, strides in elements.  Whole numbers in device memory
 * (page tables, counts, paths) are checked where they are used: none leads
 * outside the buffers named here.  They must not be written to by others while
 * a call runs.
 */
#ifndef DF11_SEARCH_H
#define DF11_SEARCH_H

#include "df11_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Attention of drafted tokens ---------------------------------------- */

/* Queries of `nodes` new tokens ("nodes") for each of `batch` sequences.  Their
 * keys and values are in the cache already: node a of sequence b at position
 * lens[b] + a (df11_paged_append wrote them). */
typedef struct df11_tree {
    const uint16_t *q;   /* BF16: node i, head g of sequence b at
                            q + b * q_batch_stride + i * q_node_stride + g * q_head_stride */
    uint64_t q_batch_stride, q_node_stride, q_head_stride;
    const int64_t *mask; /* device: bit a % 64 of word a / 64 at
                            mask + b * mask_batch_stride + i * mask_node_stride
                            says whether node i reads node a; NULL: nodes 0..i, a chain */
    uint64_t mask_batch_stride, mask_node_stride;
    const int32_t *counts; /* device: sequence b has counts[b] nodes; NULL: `nodes` */
    const int32_t *starts; /* device: node i of sequence b reads from position starts[b * starts_batch_stride +
                              i * starts_node_stride] on; NULL: from 0 */
    uint64_t starts_batch_stride, starts_node_stride;
    uint64_t batch, nodes;
    uint32_t q_heads;    /* a multiple of the cache's kv_heads; heads share keys as in df11_paged_attention */
    float scale;
} df11_tree;

/* Attention of every node over its sequence's positions [start, lens[b]), start
 * that of the node (both held to [0, table_width * page_size], start to lens),
 * and the nodes a < counts[b] that its mask names (itself only if it is named).
 * Positions past the table and table entries outside [0, n_pages) are masked;
 * page_table is as in df11_paged_attention.  With s_j = scale * q . k_j over
 * the positions that are left:
 *   out[b, i, g, :] = sum_j exp(s_j) v_j / sum_j exp(s_j)  (BF16, [batch, nodes,
 *                     q_heads, head_dim] contiguous, 16-byte aligned)
 *   lse[b, i, g]    = log sum_j exp(s_j)                   (32 bits; NULL = not wanted)
 * and zeros and -infinity where nothing is left and for nodes i >= counts[b].
 * What positions masked for a node hold, NaN and infinities included, does not
 * matter to it.  Scores, sums and the weighted values are held in 32 bits (the
 * latter may reach 256 times, with E4M3 pages 2^15 times, the sum of the values'
 * magnitudes before the division); the weights exp(s_j) enter the product as two
 * BF16 parts (16 bits) with BF16 pages, rounded to FP16 (11 bits, 2^-32 of the
 * largest at least) with E4M3 pages.  An infinity in v_j behaves as in
 * df11_paged_attention, but may give an infinity, too, where exp(s_j) is below
 * 2^-126 of the largest (there NaN).  Every sum has a fixed order.  workspace:
 * df11_paged_tree_attention_workspace_bytes bytes of device memory, 16-byte
 * aligned (NULL when that is 0), not kept between calls; calls that run at the
 * same time need one each.  batch = 0 or
 * nodes = 0 is a no-op.  Errors: DF11_E_INVALID_ARG (null or misaligned
 * pointers; sizes and strides as for df11_paged_attention, and 2^30 positions
 * or more in a table; positions of a page 256 MiB apart; mask_node_stride below
 * ceil(nodes / 64); over 2^20 nodes; 2^24 rows of the output, or 2^24
 * workgroups: batch x kv_heads x tiles of 16 to 128 rows of nodes x heads, times
 * the chunks of a sequence),
 * DF11_E_UNSUPPORTED, DF11_E_BUFFER_TOO_SMALL, DF11_E_HIP. */
df11_status df11_paged_tree_attention(const df11_paged_cache *cache, const df11_tree *tree, const int32_t *page_table,
                                      uint64_t table_stride, uint64_t table_width, const int32_t *lens, uint16_t *out,
                                      float *lse, void *workspace, uint64_t workspace_bytes, void *hip_stream);

/* Bytes of workspace for such a call (0 where positions are not split, and for calls that are refused). */
uint64_t df11_paged_tree_attention_workspace_bytes(uint64_t batch, uint64_t nodes, uint32_t q_heads, uint32_t kv_heads,
                                                   uint32_t head_dim, uint32_t page_size, uint64_t table_width);

/* ---- Pages ---------------------------------------------------------------
 * df11_paged_copy and df11_paged_compact work on the same pages of `layers`
 * layers in one call: layer l's pages start at k_pages + l * k_layer_stride and
 * v_pages + l * v_layer_stride (multiples of 16 bytes; layers up to 65535,
 * with their strides within the limit of 2^48 elements).  They move what is
 * stored bit by bit; scales are not looked at (and may be NULL). */

/* Copies the first rows[i] positions (NULL: all; held to [0, page_size]) of
 * page src[i] to page dst[i], i < n, for all heads and layers.  src, dst, rows:
 * device, 32-bit.  A pair with a page outside [0, n_pages) is skipped (padding).
 * Pairs run side by side: where a page is the target of several pairs, or of
 * one and the source of another, each 16 bytes of what is read from or left in
 * it are those of either.  n = 0 is a no-op.  Errors: DF11_E_INVALID_ARG
 * (null or misaligned pointers, n of 2^31 or more, no layers, limits above, n
 * x layers x 2 x pieces of 2^31 or more, a piece being 16 KiB of a page's K),
 * DF11_E_UNSUPPORTED (as for df11_paged_append), DF11_E_HIP. */
df11_status df11_paged_copy(const df11_paged_cache *cache, uint32_t layers, uint64_t k_layer_stride,
                            uint64_t v_layer_stride, const int32_t *src, const int32_t *dst, const int32_t *rows,
                            uint64_t n, void *hip_stream);

/* Moves what lies at positions lens[b] + path[b, i] of sequence b to lens[b] +
 * i, for i < accepted[b] (held to [0, depth]) in that order, for all heads and
 * layers: the accepted path of a drafted tree next to what the cache held.
 * path: device, 32-bit, [batch, depth] contiguous; its numbers ascend from 0 or
 * more, and the first one that does not ends the path.  A position past the
 * table or in a page outside the cache is neither read nor written: that move
 * is skipped.  lens stays as it is.  Two sequences must not move rows of one
 * page.  batch = 0 or depth = 0 is a no-op.  Errors: DF11_E_INVALID_ARG (null
 * or misaligned pointers; depth over 1024; table_width 0, or 2^31 positions or
 * more in it; table_stride below table_width; limits above; 2^31 sequences or
 * more; batch x layers x pieces of 2^31 or more, a piece
 * being 4 KiB of a position's K and V),
 * DF11_E_UNSUPPORTED, DF11_E_HIP. */
df11_status df11_paged_compact(const df11_paged_cache *cache, uint32_t layers, uint64_t k_layer_stride,
                               uint64_t v_layer_stride, const int32_t *path, uint32_t depth, const int32_t *accepted,
                               const int32_t *page_table, uint64_t table_stride, uint64_t table_width,
                               const int32_t *lens, uint64_t batch, void *hip_stream);

/* Reorders the sequences of a page table and accounts for their pages, in
 * place.  refs[p] (device, 32-bit, n_pages) counts the holders of page p: table
 * entries, and others that the caller adds (a prefix kept for later); a page
 * with 0 is free.  Row b of the new table goes on from row p = parents[b] of
 * the old one (parents NULL: p = b; outside [0, batch): row b ends).  With L =
 * lens[p] (held to [0, table_width * page_size]):
 *   columns below L / page_size  the pages of row p, shared
 *   those up to ceil((L + room) / page_size), at most table_width: if b is the
 *     lowest row that goes on from p, and refs of the page of row p was at most
 *     1, that page; otherwise a page that was free before the call
 *   all others                    -1
 * Free pages go by ascending number to the (row, column) that want one in
 * ascending order; where they run out the entry is -1 and counted in missing[0].
 * Entries outside [0, n_pages) are not pages: shared, they become -1.  A row
 * that ends becomes empty: entries -1, lens 0.  Afterwards lens[b] = L and refs
 * has every entry's change: pages that no row holds any longer are at 0 and
 * free for the next call.  Where L is no multiple of page_size and row b got a
 * free page for its last positions, src[b], dst[b], rows[b] are the old page,
 * the new one and L % page_size, otherwise -1, -1, 0: what df11_paged_copy
 * takes, for each layer, before the rows are read or appended to.
 * With parents NULL the call trims and reserves: each row holds the pages of
 * its length and of `room` more positions, and no others.
 * workspace: df11_paged_fork_workspace_bytes bytes, 16-byte aligned.  lens, refs
 * and page_table must not overlap.  Errors: DF11_E_INVALID_ARG (null or
 * misaligned pointers; batch over 4096; page_size as for a cache; table_width 0,
 * over 2^24, or 2^31 positions or more in it; table_stride below table_width or
 * over 2^32; n_pages 0 or over 2^31 - 1; room over 2^30, or with batch more than
 * 2^30 pages to be had), DF11_E_BUFFER_TOO_SMALL,
 * DF11_E_HIP.  batch = 0 sets missing[0] = 0 and nothing else. */
df11_status df11_paged_fork(const int32_t *parents, uint64_t batch, int32_t *page_table, uint64_t table_stride,
                            uint64_t table_width, uint32_t page_size, int32_t *lens, int32_t *refs, uint64_t n_pages,
                            uint64_t room, int32_t *src, int32_t *dst, int32_t *rows, int32_t *missing, void *workspace,
                            uint64_t workspace_bytes, void *hip_stream);

uint64_t df11_paged_fork_workspace_bytes(uint64_t batch, uint64_t table_width, uint32_t page_size, uint64_t n_pages,
                                         uint64_t room);

/* ---- Selection ----------------------------------------------------------- */

#define DF11_LOGITS_BF16 0u
#define DF11_LOGITS_FP32 1u

/* The k best continuations of each of `batch` searches with `beams` beams over
 * a vocabulary.  logits: BF16 bit patterns or 32-bit floats, token v of beam i
 * of search b at logits + b * batch_stride + i * beam_stride + v.  scores:
 * device, 32-bit floats [batch, beams], what the beams have so far; done: device,
 * bytes [batch, beams], nonzero for a beam that has ended (NULL: none).  A beam
 * offers, for every token v,
 *   scores[b, i] + x[v] - log sum_u exp(x[u])
 * and a beam that has ended its score as it is, once, with token `pad`.  What is
 * -infinity or NaN (a masked token, a row with NaN or +infinity, a score that is
 * no finite number) is not offered.  Best first; of equal ones the lower beam
 * first, of one beam the larger logit, then the lower token.
 *   out_scores  32-bit floats [batch, k]
 *   out_parents 32-bit [batch, k]: b * beams + i
 *   out_tokens  32-bit [batch, k]
 * Places for which nothing is left hold -infinity, -1 and `pad`.  Maxima and
 * sums of exponentials of at most 2^14 tokens are held in 32 bits, sums of those
 * and scores in 64.  workspace: as above.  batch = 0 is
 * a no-op.  Errors: DF11_E_INVALID_ARG (null or misaligned pointers; k 0 or over
 * 64; beams 0 or over 1024; vocab 0; beams * vocab of 2^31 or
 * more; batch * beams of 2^24 or more; strides over 2^40 or past 2^48 elements),
 * DF11_E_UNSUPPORTED (dtype), DF11_E_BUFFER_TOO_SMALL, DF11_E_HIP. */
df11_status df11_beam_select(const void *logits, uint32_t dtype, uint64_t batch, uint64_t beams, uint64_t vocab,
                             uint64_t batch_stride, uint64_t beam_stride, const float *scores, const uint8_t *done,
                             uint32_t k, int32_t pad, float *out_scores, int32_t *out_parents, int32_t *out_tokens,
                             void *workspace, uint64_t workspace_bytes, void *hip_stream);

uint64_t df11_beam_select_workspace_bytes(uint64_t batch, uint64_t beams, uint64_t vocab, uint32_t k);

#ifdef __cplusplus
}
#endif

#endif /* DF11_SEARCH_H */
