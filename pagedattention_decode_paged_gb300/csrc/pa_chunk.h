// pa_chunk.h -- parameter block and launchers of attention of several new
// tokens per sequence (include/pagedattn_chunk.h), shared between the C-ABI
// layer (api_chunk.cu) and the kernel translation units.
#pragma once

#include "pa_internal.h"
#include "pagedattn_chunk.h"

namespace pa {

struct ChunkParams {
    const void *q;
    int64_t q_stride;          // elements from token row to token row
    void *out;                 // [B][T][H][D]
    const char *k_pool;
    const char *v_pool;
    const int32_t *block_table;
    const int32_t *positions;
    const int32_t *counts;     // null: T for every sequence
    int32_t *err_word;
    int64_t num_blocks;
    int64_t block_stride_bytes;
    int32_t rows_per_block;    // block_stride / head_dim (tensor-map row pitch per block)
    int32_t B, T, H, Hkv, G, MB, bs;   // G = H / Hkv
    uint32_t g_mul, g_shift;   // quotients by G: chunk::by_group
    int32_t bs_shift;          // log2(bs) when bs is a power of two, else -1
    int32_t window;
    float scale_log2;          // scale * log2(e)
    // differential form: lambdas not null
    const float *lambdas;
    const void *norm_weight;
    float eps;
    float out_scale;
    // workspace: per CTA two records of the rows' softmax states, and one cut
    float *records;
    struct ChunkCut *cuts;
    int32_t rec_floats;
};

// What the second launch joins for a CTA: rows of an item that CTA w - 1 began
// and CTAs w to last went on with.
struct ChunkCut {
    int32_t b;                 // sequence; -1: nothing
    int32_t hk;                // kv head
    int32_t n0, rows;          // first of the head's rows, rows
    int32_t last;
    int32_t zeros;             // the same in all: sequences with positions out of range, whose rows the launch zeroes
    int32_t pad[2];
};

// What a kernel variant needs of the workspace on the current device.
struct ChunkPlan {
    int grid = 0;
    int rows = 0;              // query rows of an item (of each map)
    int maps = 1;
    bool two_parts = false;    // 16-bit types: weights as rounded weight and rest
    int rec_floats = 0;        // floats of a record: rows * maps of head_dim, their maxima and their sums
};
inline int chunk_rec_floats(int rows_all_maps, int head_dim) { return rows_all_maps * (head_dim + 2); }

bool chunk_supported(int dtype, int head_dim, bool diff);

// fp32 on the CUDA cores, 16-bit on mma.sync (any block size).
cudaError_t plan_chunk_f32(int head_dim, bool diff, ChunkPlan *plan);
cudaError_t launch_chunk_f32(int head_dim, const ChunkParams &p, const ChunkPlan &plan, cudaStream_t stream);
cudaError_t plan_chunk_mma(int dtype, int head_dim, bool diff, bool two_parts, ChunkPlan *plan);
cudaError_t launch_chunk_mma(int dtype, int head_dim, const ChunkParams &p, const ChunkPlan &plan, cudaStream_t stream);

// 16-bit types, head_dim 64 and 128, on tcgen05; tensor maps of the pools in
// boxes of box_rows rows, a divisor of 128 and of the block size, or box_rows 0 and
// no maps: row by row.
bool chunk_umma_supported(int dtype, int head_dim);
cudaError_t plan_chunk_umma(int dtype, int head_dim, bool diff, bool two_parts, int box_rows, ChunkPlan *plan);
// qmap: the queries in boxes of q_tokens tokens of a group's heads (q_tokens 0:
// a tile is not whole tokens, and the map is not used).
cudaError_t launch_chunk_umma(int dtype, int head_dim, const ChunkParams &p, const CUtensorMap &kmap, const CUtensorMap &vmap,
                              int box_rows, const CUtensorMap &qmap, int q_tokens, const ChunkPlan &plan,
                              cudaStream_t stream);

// A pool's tensor map in 128-byte swizzled boxes of box_rows rows (api.cu):
// head_dim 64 as [rows][64], head_dim 128 as [rows / 8][2][8][64].
bool chunk_pool_map(CUtensorMap *map, const pa_shape *s, const void *pool, int box_rows);
// The queries' tensor map: [D / 64][tokens][heads][64 elements], boxes of one
// slab of q_tokens tokens of G heads.
bool chunk_query_map(CUtensorMap *map, const pa_shape *s, const void *q, int64_t q_stride, int64_t tokens, int q_tokens);

// Join the rows that the attention kernel of `plan` left in records.
cudaError_t launch_chunk_merge(int dtype, int head_dim, const ChunkParams &p, const ChunkPlan &plan,
                               cudaStream_t stream);

}  // namespace pa
