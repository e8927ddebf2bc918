/*
 * pagedattn_fp4.h -- a paged KV cache held in 4 bits: quantising append (with
 * or without norm and rotation), decode attention, and reading rows back.
 *
 * Layouts, ownership, streams, host checks and err_word are those of
 * pagedattn.h.  The pages name quantised cache blocks ([BM] s6.3, s3) without
 * fixing a scheme; this one is:
 *
 *   A row of head_dim values is cut into groups of 16 consecutive ones.  A
 *   value is value(c) * value(s) * g, where
 *     c  is its E2M1 code (sign bit, 2 exponent bits with bias 1, 1 mantissa
 *        bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two codes to a
 *        byte, the lower element in the low four bits;
 *     s  is the group's scale, an OCP E4M3 byte (as the fp8 cache's codes);
 *     g  is one fp32 factor for all keys (k_scale), one for all values
 *        (v_scale), given with every call: 1, or what brings the largest
 *        magnitude of the cache near 6 * 448 when E4M3's range would not
 *        cover it; from 2^-64 to 2^64 (others: PA_ERR_INVALID_ARG).
 *   That is 4.5 bits per value.  The products value(c) * value(s) are exact
 *   in fp16.
 *
 *   pools      the layout of the pools of pagedattn.h with a row of
 *              head_dim/2 bytes: row (blk, kv_head, slot) starts at byte
 *                blk*block_stride + (kv_head*block_size + slot)*head_dim/2;
 *              shape->block_stride counts BYTES here, a multiple of 16
 *   kv_scales  device bytes [num_blocks][2][num_kv_heads][block_size]
 *              [head_dim/16], K's half then V's in each block, 16-byte aligned
 *
 *   shape->dtype is the type of queries, outputs and new rows (fp32, fp16 or
 *   bf16); head_dim is 64, 128 or 256 (others: PA_ERR_UNSUPPORTED).
 */
#ifndef PAGEDATTN_FP4_H
#define PAGEDATTN_FP4_H

#include "pagedattn_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * paged_kv_append_fp4 -- the quantising write of new keys and values, as
 * paged_kv_append_rope_fp4 without queries, norm and rotation (rows->q is
 * ignored).
 *
 * paged_kv_append_rope_fp4 -- paged_kv_append_rope into the 4-bit cache:
 * the queries go to q_out in the shape's dtype; each group of 16 values x of
 * a (rotated, unrounded) key or value row is written as
 *   s = E4M3(max|x| / (6 g)),   c = E2M1(x / (value(s) g)),
 * both nearest with ties to the even code and saturating (448, 6), quotients
 * and products in IEEE binary32; a NaN counts as 0, a group whose scale is 0
 * has codes 0.  Positions, counts, checks and untouched rows are those of
 * paged_kv_append_rope.
 */
pa_status paged_kv_append_fp4(const pa_shape *shape, const pa_new_rows *rows, uint8_t *k_pool,
                              uint8_t *v_pool, uint8_t *kv_scales, float k_scale, float v_scale,
                              const int32_t *block_table, const int32_t *positions,
                              const int32_t *counts, int32_t *err_word, pa_stream_t stream);

pa_status paged_kv_append_rope_fp4(const pa_shape *shape, const pa_rope *rope,
                                   const pa_new_rows *rows, void *q_out, uint8_t *k_pool,
                                   uint8_t *v_pool, uint8_t *kv_scales, float k_scale,
                                   float v_scale, const int32_t *block_table,
                                   const int32_t *positions, const int32_t *counts,
                                   int32_t *err_word, pa_stream_t stream);

/*
 * paged_kv_gather_fp4 -- read rows of the 4-bit cache back as values (a cached
 * prefix that a prompt continues, a request moving to another kind of
 * cache).
 *
 * k_out, v_out are [batch][max_tokens][num_kv_heads][head_dim] of the shape's
 * dtype: row t < counts[b] (counts NULL: max_tokens) gets the values of token
 * starts[b] + t: value(c) * value(s), exact, times g in IEEE binary32, then
 * rounded to the dtype; rows t >= counts[b] are left as they were.  num_heads
 * is not used.  counts[b] outside [0, max_tokens] gives PA_DEVERR_BAD_LEN and
 * writes nothing; starts[b] < 0 or starts[b] + counts[b] past the table row
 * gives PA_DEVERR_BAD_POS, a token whose entry is outside [0, num_blocks)
 * PA_DEVERR_BAD_BLOCK, and the rows concerned
 * are zeros.  The translation is that of [BM] s5.2.
 */
pa_status paged_kv_gather_fp4(const pa_shape *shape, void *k_out, void *v_out, int32_t max_tokens,
                              const uint8_t *k_pool, const uint8_t *v_pool,
                              const uint8_t *kv_scales, float k_scale, float v_scale,
                              const int32_t *block_table, const int32_t *starts,
                              const int32_t *counts, int32_t *err_word, pa_stream_t stream);

/*
 * paged_attention_decode_fp4 -- paged_attention_decode over the values the
 * codes stand for ([PG] s2.2), over the last `window` valid tokens when window
 * > 0 ([BUG] s5.3), on a persistent grid that gives every CTA about equal runs
 * of 32-token tiles of all (sequence, kv head) items, so that ragged batches
 * and single long contexts alike keep the whole GPU busy; an item cut between
 * CTAs is finished by the last of them (the log-sum-exp merge of the
 * split-KV pair), in a fixed order, so results repeat from call to call.
 *
 * Numerics: each head's queries are scaled by a power of two, exactly, and
 * read as fp16 (16-bit queries: exact, elements below 2^-28 of the head's
 * largest to 2^-39 of it) or as two fp16 parts (fp32: off by at most 2^-22 of
 * themselves or 2^-39 of the largest, whichever is more); keys and values are
 * exact; scores, softmax and sums are fp32; the weights enter the second
 * product in fp16, off by at most 2^-11 of themselves or 2^-32 of the largest,
 * or, with fp32 queries, as two parts: 2^-22 and 2^-32.  Device checks, zeros
 * and PA_DEVERR_* bits are those of paged_attention_decode.  A NaN scale
 * (0x7F, 0xFF) inside the attended length makes the outputs it meets NaN.
 *
 * Workspace: as for paged_attention_decode_balanced -- at least
 * paged_attention_fp4_workspace() bytes on the device, 16-byte aligned,
 * ZERO-FILLED before its first use; every call leaves its counters at zero;
 * calls that may overlap on the GPU (streams, captured graphs) need
 * workspaces of their own.  The size depends on the shape and on the current
 * device; a workspace may serve other shapes too, on the same device, if it is
 * large enough for them.  0 for a shape this entry point rejects: the schedule
 * keeps two int32 per sequence in shared memory and counts tokens and tiles in
 * int32 (PA_ERR_UNSUPPORTED: more sequences than fit, 2^30 tiles of all items,
 * or a table row of 2^31 - 1024 tokens).  8000 sequences always fit at head_dim
 * 64 and 128, 2000 at 256; a larger batch goes in several calls.  scale *
 * k_scale must be finite in fp32.
 * (The workspace query has no counterpart on the pages.)
 */
size_t paged_attention_fp4_workspace(const pa_shape *shape);

pa_status paged_attention_decode_fp4(const pa_shape *shape, void *out, const void *q,
                                     const uint8_t *k_pool, const uint8_t *v_pool,
                                     const uint8_t *kv_scales, float k_scale, float v_scale,
                                     const int32_t *block_table, const int32_t *seq_lens,
                                     float scale, int32_t window, void *workspace,
                                     size_t workspace_bytes, int32_t *err_word,
                                     pa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_FP4_H */
