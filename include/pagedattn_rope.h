/*
 * pagedattn_rope.h -- the write side of a decoder layer: per-head norm and
 * position rotation of the step's queries and keys, and the append of keys
 * and values into the paged cache, in one pass.
 *
 * Layouts, ownership, streams, host checks and err_word are those of
 * pagedattn.h.  The pages that define the cache ([BM], [KB], [BUG], [PG]
 * there) take rotated keys as given and say nothing of norms or rotation;
 * where a row goes in the cache is theirs.
 */
#ifndef PAGEDATTN_ROPE_H
#define PAGEDATTN_ROPE_H

#include "pagedattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * What happens to a query or key row x[0..head_dim) on its way, in this order:
 *   norm      (q_weight / k_weight not NULL)  y_d = (x_d * r) * w_d with
 *             r = 1 / sqrt(mean_d x_d^2 + eps), one w of head_dim elements of
 *             the shape's dtype for all heads of q, one for all heads of k
 *   rotation  (rotary_dim > 0) of the first R = rotary_dim elements in pairs
 *             (a, b): a' = a*cos - b*sin, b' = b*cos + a*sin, pair i being
 *             elements (i, i + R/2), or (2i, 2i + 1) when interleaved.
 *             Row p of cos_sin (device fp32 [max_position][R]) holds the R/2
 *             cosines, then the R/2 sines, of cache position p; elements from
 *             R on pass unchanged.
 * Value rows pass unchanged.  The arithmetic is binary32, with one rounding to
 * the target type at the end.  The norm's and the rotation's products and the
 * rotation's sums are each rounded by themselves (no fused multiply-add), so
 * that the rotation is the formula evaluated operation by operation; the mean
 * square is summed in the kernel's own order, with fused multiply-adds, before
 * eps is added and r taken with a rounding each.
 * The sum of a row's squares has to stay within binary32.  Where it passes
 * 2^128 (a root mean square of 1.6e18 at head_dim 128) r is 0 and the row
 * zeros; where every square is 0 (elements below 2^-75) and eps is 0, r is
 * infinite and the row NaN or infinities.
 * R must be a multiple of 16 not above head_dim (0: no rotation, cos_sin
 * may be NULL); cos_sin and the weights 16-byte aligned; eps >= 0 and finite
 * when there is a weight.
 */
typedef struct pa_rope {
    const float *cos_sin;
    int32_t max_position;
    int32_t rotary_dim;
    int32_t interleaved;
    const void *q_weight;
    const void *k_weight;
    float eps;
} pa_rope;

/*
 * The step's new rows, a padded batch of max_tokens tokens per sequence (1
 * for a decode step).  Token t of sequence b is row b*max_tokens + t; its
 * num_heads query rows (num_kv_heads key, value rows) of head_dim elements
 * lie one after another at q + row*q_stride (k + row*k_stride, v +
 * row*v_stride) elements, so that q, k and v may be slices of one packed
 * projection output.  A stride of 0 means rows packed without gaps; others
 * must be at least one row long.  Pointers and strides keep every row on a
 * 16-byte boundary.  q may be NULL (keys and values only, q_out is then
 * not written).
 */
typedef struct pa_new_rows {
    const void *q;
    const void *k;
    const void *v;
    int64_t q_stride;
    int64_t k_stride;
    int64_t v_stride;
    int32_t max_tokens;
} pa_new_rows;

/*
 * paged_kv_append_rope -- norm and rotate the new queries and keys, write
 * the queries to q_out and the keys and values into the cache.
 *
 * Token t < counts[b] of sequence b (counts NULL: max_tokens for all) has
 * cache position positions[b] + t: its keys are rotated for that position and
 * written, with its values, to slot pos % block_size of block
 * block_table[b][pos / block_size] ([BM] s4.4, [BUG] s4.1), as
 * paged_kv_append_tokens places them.  q_out is [batch][max_tokens][num_heads]
 * [head_dim], packed; it may be the same memory as a packed q.  Rows t >=
 * counts[b] of q_out and everything else in the pools are left as they were.
 * Two tokens that name the same slot of the pools are a caller error.
 *
 * Device checks: counts[b] outside [0, max_tokens] gives PA_DEVERR_BAD_LEN
 * and nothing of the sequence is written; positions[b] < 0, or positions[b] +
 * counts[b] past the table row or past max_position (when there is a
 * rotation) gives PA_DEVERR_BAD_POS, zeros in the sequence's counts[b] rows
 * of q_out and no write to the pools; a token whose target entry is outside
 * [0, num_blocks) gives PA_DEVERR_BAD_BLOCK and its keys and values are not
 * written (its queries are).
 *
 * Shapes: head_dim a power of two, 32..256 (16-bit) or 16..128 (fp32); others
 * give PA_ERR_UNSUPPORTED.  More than 65536 heads of a kind, or a padded batch
 * of 2^31 tokens, give PA_ERR_INVALID_ARG.  One launch on `stream`.
 */
pa_status paged_kv_append_rope(const pa_shape *shape, const pa_rope *rope, const pa_new_rows *rows,
                               void *q_out, void *k_pool, void *v_pool,
                               const int32_t *block_table, const int32_t *positions,
                               const int32_t *counts, int32_t *err_word, pa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_ROPE_H */
