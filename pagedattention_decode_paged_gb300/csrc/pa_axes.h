// pa_axes.h -- parameter block and launcher of the rotary append with positions
// of several axes (include/pagedattn_axes.h).
#pragma once

#include "pa_rope_fp4.h"
#include "pagedattn_axes.h"

namespace pa {

struct RopeAxesParams : RopeAppendParams {
    const int32_t *axis_positions;   // [axes][B][T]
    int32_t axes;
    uint8_t pair_axis[32];     // axis of pair i in bits 2 (i % 4) of byte i / 4
};

cudaError_t launch_rope_append_axes(int dtype, int head_dim, const RopeAxesParams &p, cudaStream_t stream);

}  // namespace pa
