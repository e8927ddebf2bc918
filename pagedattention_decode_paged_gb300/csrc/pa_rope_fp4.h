// pa_rope_fp4.h -- parameter blocks and launchers of the rotary append and the
// 4-bit cache (include/pagedattn_rope.h, include/pagedattn_fp4.h), shared
// between the C-ABI layer (api_rope_fp4.cu) and the kernel translation units.
#pragma once

#include "pa_internal.h"
#include "pagedattn_fp4.h"
#include "pagedattn_rope.h"

namespace pa {

struct RopeAppendParams {
    const void *q;             // null: keys and values only
    const void *k;
    const void *v;
    int64_t q_stride, k_stride, v_stride;   // elements from token row to token row
    void *q_out;               // [B][T][H][D]
    char *k_pool;
    char *v_pool;
    uint8_t *scales;           // 4-bit cache: E4M3 scales [NB][2][Hkv][bs][D/16]
    const int32_t *block_table;
    const int32_t *positions;
    const int32_t *counts;     // null: T for every sequence
    int32_t *err_word;
    const float *cos_sin;      // [max_position][R]
    const void *q_weight;
    const void *k_weight;
    int64_t num_blocks;
    int64_t block_stride_bytes;
    int32_t B, T, H, Hkv, MB, bs;
    int32_t bs_shift;          // log2(bs) when bs is a power of two, else -1
    int32_t max_position, R, pairs;
    float eps;
    float k_g, v_g;
};

// fp4: write the 4-bit cache (fp4_head_dim), else a cache of `dtype` (rope_append_supported).
bool rope_append_supported(int dtype, int head_dim);
cudaError_t launch_rope_append(int dtype, int head_dim, bool fp4, const RopeAppendParams &p, cudaStream_t stream);

struct GatherFp4Params {
    void *k_out;
    void *v_out;
    const uint8_t *k_pool;
    const uint8_t *v_pool;
    const uint8_t *scales;
    const int32_t *block_table;
    const int32_t *starts;
    const int32_t *counts;
    int32_t *err_word;
    int64_t num_blocks;
    int64_t block_stride_bytes;
    int32_t B, T, Hkv, MB, bs;
    int32_t bs_shift;
    float k_g, v_g;
};

cudaError_t launch_gather_fp4(int dtype, int head_dim, const GatherFp4Params &p, cudaStream_t stream);

inline bool fp4_head_dim(int head_dim) { return head_dim == 64 || head_dim == 128 || head_dim == 256; }

// Decode over the 4-bit cache.  DecodeParams as for the balanced kernels
// (final mode, plain or window); block_stride_bytes in bytes of the pools.
struct Fp4Decode {
    DecodeParams d;
    const uint8_t *scales;
    float v_g;                 // factor of all values (k_scale is folded into d.scale_log2)
};

// A plan fixes the grid for a shape on the current device.  The workspace
// holds 4 records of kFp4RecFloats floats and two int32 group counters for each
// CTA of the largest grid, then one int32 counter per item.
constexpr int kFp4RecFloats = 16 * 128 + 2 * 16;   // the largest item: 16 heads of 128
struct Fp4Plan {
    int grid = 0;
    int max_grid = 0;          // of any shape on this device
    size_t smem = 0;
    int units_per_kv = 1;      // items per (sequence, kv head)
    int nt = 1;                // 8-column MMA tiles per item
    bool whole_tiles = false;  // the rows of a tile are contiguous
    int64_t items = 0;
};
cudaError_t plan_decode_fp4(int dtype, int head_dim, int group, int batch, int kv_heads, int block_size,
                            int64_t max_tiles_per_item, Fp4Plan *plan);
cudaError_t launch_decode_fp4(int dtype, const Fp4Decode &p, const Fp4Plan &plan, cudaStream_t stream);

}  // namespace pa
