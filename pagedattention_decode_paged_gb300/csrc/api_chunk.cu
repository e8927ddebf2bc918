// api_chunk.cu -- the extern "C" entry points of include/pagedattn_chunk.h:
// host-side validation, kernel selection and launches.  Nothing here allocates
// device memory or synchronises the host.
#include <math.h>

#include <algorithm>

#include "pa_chunk.h"

namespace pa {

bool chunk_supported(int dtype, int head_dim, bool diff) {
    if (dtype == PA_F32) return (head_dim == 16 && !diff) || head_dim == 32 || head_dim == 64 || head_dim == 128;
    return head_dim == 32 || head_dim == 64 || head_dim == 128 || head_dim == 256;
}

}  // namespace pa

namespace {

int elem_size(int32_t dtype) { return dtype == PA_F32 ? 4 : 2; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pa_status check_shape(const pa_shape *s, bool diff) {
    if (s == nullptr) return PA_ERR_INVALID_ARG;
    if (s->dtype != PA_F32 && s->dtype != PA_F16 && s->dtype != PA_BF16) return PA_ERR_INVALID_ARG;
    if (s->batch < 0 || s->num_heads <= 0 || s->num_kv_heads <= 0 || s->head_dim <= 0 || s->block_size <= 0 ||
        s->max_blocks_per_seq <= 0 || s->num_blocks <= 0)
        return PA_ERR_INVALID_ARG;
    if (s->num_heads % s->num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    if (!pa::chunk_supported(s->dtype, s->head_dim, diff)) return PA_ERR_UNSUPPORTED;
    if (s->block_stride < (int64_t)s->num_kv_heads * s->block_size * s->head_dim) return PA_ERR_INVALID_ARG;
    const int64_t max_len = (int64_t)s->max_blocks_per_seq * s->block_size;
    if (max_len > INT32_MAX) return PA_ERR_INVALID_ARG;
    if (max_len > INT32_MAX - 1024) return PA_ERR_UNSUPPORTED;   // a tile past the last position stays in int32
    if (s->block_stride * elem_size(s->dtype) % 16 != 0) return PA_ERR_MISALIGNED;
    return PA_OK;
}

// Rows of the tcgen05 kernel's boxes: what divides a tile of 128 positions and a
// block; 0 where the pool does not fit them (rows of a block in whole groups of
// 8, TMA row coordinates in int32): rows are copied one by one then.
int umma_box_rows(const pa_shape *s) {
    if (s->block_size % 8 != 0) return 0;
    if (s->block_stride % (8 * s->head_dim) != 0) return 0;
    if (s->num_blocks > (int64_t)INT32_MAX / (s->block_stride / s->head_dim)) return 0;
    int rows = 128;
    while (s->block_size % rows != 0) rows /= 2;
    return rows;
}

// Row by row, one warp of the tcgen05 kernel's CTA copies K and V; on mma.sync the
// four of each of up to seven CTAs do.  Query rows of a kv head (tokens of the padded
// batch times heads of the group) above which the products outweigh that.  tcgen05
// against mma.sync, fp16, one part of weights (two, as up to 128 rows have them, add a
// tenth on mma.sync), behind 2047 tokens: 32 sequences, 64 heads on 8 of 128, blocks
// of 1: 8 rows 178 and 96 us, 64 rows 195 and 108, 128 rows 202 and 196, 256 rows 218
// and 367; 16 sequences, 32 heads on 8 of 64, blocks of 3: 128 rows 82 and 64, 256 rows 91
// and 111; 32 heads of 128: 128 rows 403 and 368, 256 rows 445 and 724; behind none 128
// rows 26 and 20, 16 and 11, 42 and 42, 256 rows 29 and 35, 17 and 16, 78 and 92.  Of one
// kv head in 4 sequences there is too little for either (256 rows 29 and 27).  The host
// knows the padded batch, not the counts: a step of one piece of 512 tokens beside 63
// single ones over blocks of 1 takes tcgen05's 541 us for 525.
constexpr int kRowsAbove = 128;

// Query rows of a kv head (tokens of the padded batch times heads of the group) up to
// which weights are held in two parts, so that single and speculative tokens come out as
// exact as from the decode of the same cache (32 single tokens behind 2047, 64 heads on 8
// of 128: errors of 1.0 times the rounding of an exact result, 1.35 to 1.4 with one part).
// They mostly wait for memory (7 to 9% for the second part; 64 of 32 heads without
// groups, 128 rows multiplied for each, 28%); prompts would wait for the products (24 to
// 33%).  By the call, not by the sequence: a kernel with both forms takes 480 us for the
// 422 of 8 prompts of 900 to 2047 tokens, and 199 for 159 where single tokens are mixed
// with pieces of prompts.
constexpr int kRowsInTwoParts = 128;
static_assert(kRowsInTwoParts <= kRowsAbove, "no kernel has two parts of the plain form row by row");
bool two_parts(const pa_shape *s, bool diff, int64_t rows) {
    return diff || (s->dtype != PA_F32 && rows <= kRowsInTwoParts);
}

// The kernel for a call, and its plan on the current device.
enum Kernel { kF32, kMma, kUmma };
struct Choice {
    Kernel kernel;
    int box_rows = 0;
    bool two_parts = false;
    pa::ChunkPlan plan;
};
cudaError_t plan(const pa_shape *s, bool diff, Choice *c) {
    if (c->kernel == kF32) return pa::plan_chunk_f32(s->head_dim, diff, &c->plan);
    if (c->kernel == kMma) return pa::plan_chunk_mma(s->dtype, s->head_dim, diff, c->two_parts, &c->plan);
    return pa::plan_chunk_umma(s->dtype, s->head_dim, diff, c->two_parts, c->box_rows, &c->plan);
}
cudaError_t choose(const pa_shape *s, bool diff, float scale_log2, int64_t rows, Choice *c) {
    c->kernel = s->dtype == PA_F32 ? kF32 : kMma;
    c->two_parts = two_parts(s, diff, rows);
    // the tcgen05 kernel takes the maximum before it scales
    if (s->dtype != PA_F32 && pa::chunk_umma_supported(s->dtype, s->head_dim) && scale_log2 > 0.f) {
        c->box_rows = umma_box_rows(s);
        if (c->box_rows > 0 || rows > kRowsAbove) c->kernel = kUmma;
    }
    return plan(s, diff, c);
}
cudaError_t launch(const pa_shape *s, const pa::ChunkParams &p, const Choice &c, cudaStream_t stream) {
    if (c.kernel == kF32) return pa::launch_chunk_f32(s->head_dim, p, c.plan, stream);
    if (c.kernel == kMma) return pa::launch_chunk_mma(s->dtype, s->head_dim, p, c.plan, stream);
    CUtensorMap kmap{}, vmap{};
    if (c.box_rows > 0 && (!pa::chunk_pool_map(&kmap, s, p.k_pool, c.box_rows) || !pa::chunk_pool_map(&vmap, s, p.v_pool, c.box_rows)))
        return cudaErrorInvalidValue;
    // a tile of 128 rows is whole tokens; no more of them than there are
    CUtensorMap qmap{};
    int q_tokens = 128 % p.G == 0 ? std::min(128 / p.G, p.T) : 0;
    if (q_tokens > 0 && (p.q_stride * 2 >= (int64_t)1 << 40 ||
                         !pa::chunk_query_map(&qmap, s, p.q, p.q_stride, (int64_t)p.B * p.T, q_tokens)))
        q_tokens = 0;
    return pa::launch_chunk_umma(s->dtype, s->head_dim, p, kmap, vmap, c.box_rows, qmap, q_tokens, c.plan, stream);
}

// Two records per CTA, then its cut.
size_t cuts_at(const pa::ChunkPlan &plan) { return ((size_t)2 * plan.grid * plan.rec_floats * 4 + 15) & ~(size_t)15; }
size_t ws_bytes(const pa::ChunkPlan &plan) { return cuts_at(plan) + (size_t)plan.grid * sizeof(pa::ChunkCut); }

pa_status run(const pa_shape *s, const pa_diff *diff, void *out, const void *q, int64_t q_stride, int32_t max_tokens,
              const void *k_pool, const void *v_pool, const int32_t *block_table, const int32_t *positions,
              const int32_t *counts, float scale, int32_t window, void *workspace, size_t workspace_bytes,
              int32_t *err_word, pa_stream_t stream) {
    pa_status st = check_shape(s, diff != nullptr);
    if (st != PA_OK) return st;
    if (max_tokens < 0 || window < 0 || !isfinite(scale)) return PA_ERR_INVALID_ARG;
    const float scale_log2 = (float)((double)scale * 1.4426950408889634);
    if (!isfinite(scale_log2)) return PA_ERR_INVALID_ARG;
    if (diff != nullptr) {
        if (!isfinite(diff->out_scale)) return PA_ERR_INVALID_ARG;
        if (diff->norm_weight != nullptr && !(isfinite(diff->eps) && diff->eps >= 0.f)) return PA_ERR_INVALID_ARG;
        if (!aligned16(diff->norm_weight)) return PA_ERR_MISALIGNED;
    }
    const int es = elem_size(s->dtype), G = s->num_heads / s->num_kv_heads;
    const int64_t q_row = (int64_t)s->num_heads * s->head_dim, qs = q_stride != 0 ? q_stride : q_row;
    if (qs < q_row) return PA_ERR_INVALID_ARG;
    if ((int64_t)s->batch * max_tokens > INT32_MAX) return PA_ERR_INVALID_ARG;
    if ((int64_t)max_tokens * G > INT32_MAX - 1024) return PA_ERR_UNSUPPORTED;
    if (s->batch == 0 || max_tokens == 0) return PA_OK;
    if (out == nullptr || q == nullptr || k_pool == nullptr || v_pool == nullptr || block_table == nullptr ||
        positions == nullptr || workspace == nullptr || (diff != nullptr && diff->lambdas == nullptr))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || qs * es % 16 != 0 || !aligned16(k_pool) || !aligned16(v_pool) ||
        !aligned16(workspace))
        return PA_ERR_MISALIGNED;
    Choice c;
    if (choose(s, diff != nullptr, scale_log2, (int64_t)max_tokens * G, &c) != cudaSuccess) return PA_ERR_CUDA;
    const pa::ChunkPlan &plan = c.plan;
    if (workspace_bytes < ws_bytes(plan)) return PA_ERR_WORKSPACE;
    pa::ChunkParams p{};
    p.q = q;
    p.q_stride = qs;
    p.out = out;
    p.k_pool = static_cast<const char *>(k_pool);
    p.v_pool = static_cast<const char *>(v_pool);
    p.block_table = block_table;
    p.positions = positions;
    p.counts = counts;
    p.err_word = err_word;
    p.num_blocks = s->num_blocks;
    p.block_stride_bytes = s->block_stride * es;
    p.rows_per_block = (int32_t)(s->block_stride / s->head_dim);
    p.B = s->batch;
    p.T = max_tokens;
    p.H = s->num_heads;
    p.Hkv = s->num_kv_heads;
    p.G = G;
    for (p.g_shift = 0; (int64_t)1 << p.g_shift < G;) ++p.g_shift;
    p.g_mul = (uint32_t)((((uint64_t)1 << (31 + p.g_shift)) + G - 1) / G);
    p.MB = s->max_blocks_per_seq;
    p.bs = s->block_size;
    p.bs_shift = -1;
    for (int sh = 0; sh < 31; ++sh)
        if ((1 << sh) == s->block_size) p.bs_shift = sh;
    p.window = window;
    p.scale_log2 = scale_log2;
    if (diff != nullptr) {
        p.lambdas = diff->lambdas;
        p.norm_weight = diff->norm_weight;
        p.eps = diff->eps;
        p.out_scale = diff->out_scale;
    }
    p.records = static_cast<float *>(workspace);
    p.cuts = reinterpret_cast<pa::ChunkCut *>(static_cast<char *>(workspace) + cuts_at(plan));
    p.rec_floats = plan.rec_floats;
    const cudaStream_t on = reinterpret_cast<cudaStream_t>(stream);
    if (launch(s, p, c, on) != cudaSuccess) return PA_ERR_CUDA;
    return pa::launch_chunk_merge(s->dtype, s->head_dim, p, plan, on) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t paged_attention_chunk_workspace(const pa_shape *shape) {
    if (check_shape(shape, false) != PA_OK || shape->batch == 0) return 0;
    size_t n = 0;
    for (int i = 0; i < 8; ++i) {              // every kernel that may be chosen: of many rows and of few, with
        Choice c;                              // and without a second map
        const bool diff = i & 1;
        const int64_t rows = i & 2 ? kRowsInTwoParts : INT32_MAX;
        c.kernel = shape->dtype == PA_F32 ? kF32 : i < 4 ? kMma : kUmma;
        c.two_parts = two_parts(shape, diff, rows);
        if (!pa::chunk_supported(shape->dtype, shape->head_dim, diff)) continue;
        if (c.kernel == kUmma) {
            if (!pa::chunk_umma_supported(shape->dtype, shape->head_dim)) continue;
            c.box_rows = umma_box_rows(shape);
            if (c.box_rows == 0 && rows <= kRowsAbove) continue;
        }
        if (plan(shape, diff, &c) != cudaSuccess) return 0;
        n = std::max(n, ws_bytes(c.plan));
    }
    return n;
}

pa_status paged_attention_chunk(const pa_shape *shape, void *out, const void *q, int64_t q_stride,
                                int32_t max_tokens, const void *k_pool, const void *v_pool,
                                const int32_t *block_table, const int32_t *positions,
                                const int32_t *counts, float scale, int32_t window, void *workspace,
                                size_t workspace_bytes, int32_t *err_word, pa_stream_t stream) {
    return run(shape, nullptr, out, q, q_stride, max_tokens, k_pool, v_pool, block_table, positions, counts, scale,
               window, workspace, workspace_bytes, err_word, stream);
}

pa_status paged_attention_chunk_diff(const pa_shape *shape, const pa_diff *diff, void *out,
                                     const void *q, int64_t q_stride, int32_t max_tokens,
                                     const void *k_pool, const void *v_pool,
                                     const int32_t *block_table, const int32_t *positions,
                                     const int32_t *counts, float scale, int32_t window,
                                     void *workspace, size_t workspace_bytes, int32_t *err_word,
                                     pa_stream_t stream) {
    if (diff == nullptr) return PA_ERR_INVALID_ARG;
    return run(shape, diff, out, q, q_stride, max_tokens, k_pool, v_pool, block_table, positions, counts, scale, window,
               workspace, workspace_bytes, err_word, stream);
}

}  // extern "C"
