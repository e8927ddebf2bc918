/*
 * pagedattn_chunk.h -- attention of several new tokens per sequence over the
 * paged cache: whole prompts, pieces of long ones, speculative tokens, single
 * tokens, and batches that mix them; and the same with the difference of two
 * softmax maps.
 *
 * Layouts, ownership, streams, host checks and err_word are those of
 * pagedattn.h.  The pages that define the cache ([BM], [KB], [BUG], [PG]
 * there) attend with one token at a time; where a cached row lies ([BM] s5.2),
 * that only valid rows count ([BUG] s2.4) and the arithmetic ([PG] s2.2) are
 * theirs, the mask among the new tokens is stated here.
 */
#ifndef PAGEDATTN_CHUNK_H
#define PAGEDATTN_CHUNK_H

#include "pagedattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The new tokens are a padded batch of max_tokens tokens per sequence, as in
 * pagedattn_rope.h: token t of sequence b is row b*max_tokens + t, and its
 * num_heads query rows of head_dim elements lie one after another at
 * q + row*q_stride elements (0: rows packed without gaps; others at least one
 * row long), so that q may be a slice of a packed projection output.  out is
 * [batch][max_tokens][num_heads][head_dim], packed, and may not overlap q.
 *
 * Token t < counts[b] (counts NULL: max_tokens for all) has cache position
 * p = positions[b] + t; its own key and value and all before it are in the
 * cache already (paged_kv_append_rope and paged_kv_append_tokens put them
 * there with the same positions and counts).  It attends to the positions
 * max(0, p - window + 1) .. p, with window 0 to all of 0 .. p:
 *   out = sum_j w_j V[j] / sum_j w_j,  w_j = exp(x_j - max x),
 *   x_j = scale * <q, K[j]>,
 * so that with max_tokens 1 and positions = seq_lens - 1 it is
 * paged_attention_decode or, windowed, paged_attention_decode_window: mostly the
 * faster calls for a step of single tokens alone (64 heads on 8 of 128, bf16,
 * 32 behind 2047: 46 us for 62 here; 1 behind 131071 167 for 108, and 32 over
 * blocks of 1 843 for 106).
 * Rows t >= counts[b] of out are left as they were.  What lies in the cache
 * outside a token's positions does not reach its rows, not even as a NaN.
 *
 * Device checks: counts[b] outside [0, max_tokens] gives PA_DEVERR_BAD_LEN
 * and nothing of the sequence is written; positions[b] < 0 or positions[b] +
 * counts[b] past the table row gives PA_DEVERR_BAD_POS and zeros in the
 * sequence's counts[b] rows; a table entry outside [0, num_blocks) among
 * those of the positions that a token attends to gives PA_DEVERR_BAD_BLOCK
 * and zeros in that token's rows.
 *
 * Schedule: a persistent grid whose CTAs take equal runs of the tiles of all
 * (sequence, kv head, run of query rows), so that ragged batches, single long
 * contexts and mixes of both keep the whole GPU busy; rows whose positions are
 * cut between CTAs are joined by a second small launch (the log-sum-exp merge
 * of the split-KV pair), in a fixed order: results repeat from call to call.
 *
 * Numerics: scores, softmax and sums are fp32, and so are the products of the
 * fp32 type.  With 16-bit types the weights enter the second product rounded
 * to the type, each off by at most half a step of itself (2^-8 for bf16, 2^-11
 * for fp16, or 2^-25 of the largest), and what they were rounded to is what the
 * rows are normalised by.  In the differential form, and in calls of at most
 * 128 query rows of a kv head (max_tokens * num_heads / num_kv_heads: single
 * and speculative tokens, which so come out as exact as from
 * paged_attention_decode), they enter as two parts, off by the square of that
 * (2^-16; 2^-22, or 2^-25 of the largest).
 *
 * Workspace: at least paged_attention_chunk_workspace() bytes on the device,
 * 16-byte aligned, of any content; nothing in it is kept from call to call.
 * Calls that may overlap on the GPU (streams, captured graphs) need
 * workspaces of their own.  The size depends on the shape (batch, heads and
 * tables of any size share one) and on the current device; 0 for a shape that
 * the entry points reject or that has no sequences.
 * (The workspace query has no counterpart on the pages.)
 *
 * Shapes: head_dim 32, 64, 128 or 256 (16-bit) or 16, 32, 64 or 128 (fp32);
 * others, or 2^31 query rows of one kv head (max_tokens * num_heads /
 * num_kv_heads), or a table row of 2^31 - 1024 tokens, give
 * PA_ERR_UNSUPPORTED.  Two launches on `stream`.
 */
size_t paged_attention_chunk_workspace(const pa_shape *shape);

pa_status paged_attention_chunk(const pa_shape *shape, void *out, const void *q, int64_t q_stride,
                                int32_t max_tokens, const void *k_pool, const void *v_pool,
                                const int32_t *block_table, const int32_t *positions,
                                const int32_t *counts, float scale, int32_t window, void *workspace,
                                size_t workspace_bytes, int32_t *err_word, pa_stream_t stream);

/*
 * paged_attention_chunk_diff -- differential attention: with E = head_dim, a
 * key row of the cache holds the key of the first map in its elements
 * [0, E/2) and that of the second in [E/2, E), and so does a query row;
 * values and outputs have E elements.  For query head h
 *   a_m = softmax over the attended j of scale * <q_m, K_m[j]>   (m = 1, 2)
 *   o   = sum_j (a_1j - lambdas[h] * a_2j) V[j]
 *   y   = o * r * norm_weight,  r = 1 / sqrt(mean_d o_d^2 + eps)
 *         (norm_weight NULL: y = o)
 *   out = y * out_scale
 * lambdas: device fp32 [num_heads]; norm_weight: E elements of the shape's
 * dtype for all heads, 16-byte aligned; eps >= 0 and finite when there is a
 * weight; out_scale finite.  The two sums are taken apart, so where a V[j] is
 * infinite o may be NaN.  The squares of o_d and their sum are fp32: where it
 * passes 2^128, r is 0; where every square is 0 and eps is 0, r is infinite and
 * the row NaN or infinities.  Everything else is as for paged_attention_chunk,
 * the workspace included; zeros stay zeros.  head_dim is 32, 64, 128 or 256
 * (16-bit) or 32, 64 or 128 (fp32).  scale is usually 1/sqrt(E/2).
 * (The pages have no differential heads: the form is stated here.)
 */
typedef struct pa_diff {
    const float *lambdas;
    const void *norm_weight;
    float eps;
    float out_scale;
} pa_diff;

pa_status paged_attention_chunk_diff(const pa_shape *shape, const pa_diff *diff, void *out,
                                     const void *q, int64_t q_stride, int32_t max_tokens,
                                     const void *k_pool, const void *v_pool,
                                     const int32_t *block_table, const int32_t *positions,
                                     const int32_t *counts, float scale, int32_t window,
                                     void *workspace, size_t workspace_bytes, int32_t *err_word,
                                     pa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_CHUNK_H */
