/*
 * pagedattn_axes.h -- the rotary append of pagedattn_rope.h for tokens with
 * positions on several axes (image and video patches among text).
 */
#ifndef PAGEDATTN_AXES_H
#define PAGEDATTN_AXES_H

#include "pagedattn_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * paged_kv_append_rope_axes -- paged_kv_append_rope for tokens with positions
 * on several axes (time, row and column of an image or video patch; text has
 * the same one on each).
 *
 * Pair i of the rotation turns by the token's position on axis pair_axis[i],
 * a = positions[pair_axis[i]][b][t] of the axes: its cosine and sine are
 * cos_sin[a][i] and cos_sin[a][R/2 + i].  pair_axis is a HOST array of
 * rotary_dim/2 values below num_axes (1 to 4), read before the call returns:
 * sections of pairs, axes in turn, or any other division.  The axes' positions
 * are device int32 [num_axes][batch][max_tokens]; those of tokens t >=
 * counts[b] are not used.  Where a token's rows go in the cache is still
 * positions[b] + t, which max_position does not bound here: a token with an
 * axis position outside [0, max_position) gives PA_DEVERR_BAD_POS, zeros in
 * its rows of q_out and no write to the pools.  rotary_dim must be positive.
 * Everything else is as for paged_kv_append_rope; equal positions on all axes
 * give its results bit for bit.
 * (The pages have no rotation: the form is stated here.)
 */
typedef struct pa_rope_axes {
    const int32_t *positions;
    int32_t num_axes;
    const uint8_t *pair_axis;
} pa_rope_axes;

pa_status paged_kv_append_rope_axes(const pa_shape *shape, const pa_rope *rope,
                                    const pa_rope_axes *axes, const pa_new_rows *rows, void *q_out,
                                    void *k_pool, void *v_pool, const int32_t *block_table,
                                    const int32_t *positions, const int32_t *counts,
                                    int32_t *err_word, pa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_AXES_H */
