// api_rope_fp4.cu -- the extern "C" entry points of include/pagedattn_rope.h,
// include/pagedattn_axes.h and include/pagedattn_fp4.h: host-side validation and launches.  Nothing
// here allocates device memory or synchronises the host.
#include <math.h>

#include "pa_axes.h"

namespace {

int elem_size(int32_t dtype) { return dtype == PA_F32 ? 4 : 2; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// far enough inside fp32 that no scale times factor over- or underflows
bool factor_ok(float g) { return g >= 0x1p-64f && g <= 0x1p64f; }

// log2 of a power of two, else -1
int32_t log2_or_none(int32_t n) {
    for (int sh = 0; sh < 31; ++sh)
        if ((1 << sh) == n) return sh;
    return -1;
}

// Sizes common to every entry point; `row_bytes`: bytes of a cache row,
// `stride_bytes`: block_stride in bytes.
pa_status check_sizes(const pa_shape *s, int64_t row_bytes, int64_t stride_bytes) {
    if (s->batch < 0 || s->num_heads <= 0 || s->num_kv_heads <= 0 || s->block_size <= 0 ||
        s->max_blocks_per_seq <= 0 || s->num_blocks <= 0)
        return PA_ERR_INVALID_ARG;
    // positions and lengths are int32: the row must address fewer than 2^31 tokens
    if ((int64_t)s->max_blocks_per_seq * s->block_size > INT32_MAX) return PA_ERR_INVALID_ARG;
    if (s->num_heads > 65536 || s->num_kv_heads > 65536) return PA_ERR_INVALID_ARG;   // the grid's second axis holds them
    if (stride_bytes < (int64_t)s->num_kv_heads * s->block_size * row_bytes) return PA_ERR_INVALID_ARG;
    if (stride_bytes % 16 != 0) return PA_ERR_MISALIGNED;
    return PA_OK;
}

pa_status check_type(const pa_shape *s) {
    if (s == nullptr) return PA_ERR_INVALID_ARG;
    if (s->dtype != PA_F32 && s->dtype != PA_F16 && s->dtype != PA_BF16) return PA_ERR_INVALID_ARG;
    if (s->head_dim <= 0) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

pa_status check_fp4_shape(const pa_shape *s, bool grouped) {
    pa_status st = check_type(s);
    if (st != PA_OK) return st;
    if (!pa::fp4_head_dim(s->head_dim)) return PA_ERR_UNSUPPORTED;
    st = check_sizes(s, s->head_dim / 2, s->block_stride);
    if (st != PA_OK) return st;
    return grouped && s->num_heads % s->num_kv_heads != 0 ? PA_ERR_INVALID_ARG : PA_OK;
}

// The append entry points: `rope` null without norm and rotation, `axes` null
// for positions of one axis, `fp4` the 4-bit cache (kv_scales, k_g, v_g).
pa_status append(const pa_shape *s, const pa_rope *rope, const pa_rope_axes *axes, const pa_new_rows *rows, bool with_q,
                 void *q_out,
                 void *k_pool, void *v_pool, bool fp4, uint8_t *kv_scales, float k_g, float v_g,
                 const int32_t *block_table, const int32_t *positions, const int32_t *counts, int32_t *err_word,
                 pa_stream_t stream) {
    pa_status st = check_type(s);
    if (st != PA_OK) return st;
    if (fp4) {
        st = check_fp4_shape(s, false);
    } else {
        if (!pa::rope_append_supported(s->dtype, s->head_dim)) return PA_ERR_UNSUPPORTED;
        st = check_sizes(s, (int64_t)s->head_dim * elem_size(s->dtype), s->block_stride * elem_size(s->dtype));
    }
    if (st != PA_OK) return st;
    if (rows == nullptr || rows->max_tokens < 0) return PA_ERR_INVALID_ARG;
    if (rope != nullptr) {
        if (rope->rotary_dim < 0 || rope->rotary_dim > s->head_dim || rope->rotary_dim % 16 != 0)
            return PA_ERR_INVALID_ARG;
        if (rope->rotary_dim > 0 && (rope->cos_sin == nullptr || rope->max_position <= 0)) return PA_ERR_INVALID_ARG;
        const bool norm = rope->q_weight != nullptr || rope->k_weight != nullptr;
        if (norm && !(isfinite(rope->eps) && rope->eps >= 0.f)) return PA_ERR_INVALID_ARG;
        if (!aligned16(rope->cos_sin) || !aligned16(rope->q_weight) || !aligned16(rope->k_weight))
            return PA_ERR_MISALIGNED;
    }
    if (axes != nullptr) {
        if (rope->rotary_dim == 0 || axes->num_axes < 1 || axes->num_axes > 4 || axes->pair_axis == nullptr)
            return PA_ERR_INVALID_ARG;
        for (int i = 0; i < rope->rotary_dim / 2; ++i)
            if (axes->pair_axis[i] >= axes->num_axes) return PA_ERR_INVALID_ARG;
    }
    if (fp4 && (!factor_ok(k_g) || !factor_ok(v_g))) return PA_ERR_INVALID_ARG;
    const int es = elem_size(s->dtype);
    const bool q = with_q && rows->q != nullptr;
    const int64_t q_row = (int64_t)s->num_heads * s->head_dim, kv_row = (int64_t)s->num_kv_heads * s->head_dim;
    const int64_t qs = rows->q_stride != 0 ? rows->q_stride : q_row;
    const int64_t ks = rows->k_stride != 0 ? rows->k_stride : kv_row;
    const int64_t vs = rows->v_stride != 0 ? rows->v_stride : kv_row;
    if ((q && qs < q_row) || ks < kv_row || vs < kv_row) return PA_ERR_INVALID_ARG;
    if ((int64_t)s->batch * rows->max_tokens > INT32_MAX) return PA_ERR_INVALID_ARG;
    if (s->batch == 0 || rows->max_tokens == 0) return PA_OK;
    if (rows->k == nullptr || rows->v == nullptr || k_pool == nullptr || v_pool == nullptr ||
        block_table == nullptr || positions == nullptr || (q && q_out == nullptr) || (fp4 && kv_scales == nullptr) ||
        (axes != nullptr && axes->positions == nullptr))
        return PA_ERR_INVALID_ARG;
    if ((q && (!aligned16(rows->q) || !aligned16(q_out) || qs * es % 16 != 0)) || !aligned16(rows->k) ||
        !aligned16(rows->v) || ks * es % 16 != 0 || vs * es % 16 != 0 || !aligned16(k_pool) || !aligned16(v_pool) ||
        (fp4 && !aligned16(kv_scales)))
        return PA_ERR_MISALIGNED;
    pa::RopeAxesParams p{};
    p.q = q ? rows->q : nullptr;
    p.k = rows->k;
    p.v = rows->v;
    p.q_stride = qs;
    p.k_stride = ks;
    p.v_stride = vs;
    p.q_out = q_out;
    p.k_pool = static_cast<char *>(k_pool);
    p.v_pool = static_cast<char *>(v_pool);
    p.scales = kv_scales;
    p.block_table = block_table;
    p.positions = positions;
    p.counts = counts;
    p.err_word = err_word;
    p.num_blocks = s->num_blocks;
    p.block_stride_bytes = fp4 ? s->block_stride : s->block_stride * es;
    p.B = s->batch;
    p.T = rows->max_tokens;
    p.H = s->num_heads;
    p.Hkv = s->num_kv_heads;
    p.MB = s->max_blocks_per_seq;
    p.bs = s->block_size;
    p.bs_shift = log2_or_none(s->block_size);
    if (rope != nullptr) {
        p.cos_sin = rope->cos_sin;
        p.max_position = rope->max_position;
        p.R = rope->rotary_dim;
        p.pairs = rope->interleaved != 0;
        p.q_weight = rope->q_weight;
        p.k_weight = rope->k_weight;
        p.eps = rope->eps;
    }
    p.k_g = k_g;
    p.v_g = v_g;
    if (axes != nullptr) {
        p.axis_positions = axes->positions;
        p.axes = axes->num_axes;
        for (int i = 0; i < rope->rotary_dim / 2; ++i) p.pair_axis[i / 4] |= (uint8_t)(axes->pair_axis[i] << 2 * (i % 4));
        return pa::launch_rope_append_axes(s->dtype, s->head_dim, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? PA_OK
                   : PA_ERR_CUDA;
    }
    return pa::launch_rope_append(s->dtype, s->head_dim, fp4, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

// The decode schedule for `s` on the current device.
pa_status plan_of(const pa_shape *s, pa::Fp4Plan *plan) {
    const int64_t max_len = (int64_t)s->max_blocks_per_seq * s->block_size;
    if (max_len > INT32_MAX - 1024) return PA_ERR_UNSUPPORTED;   // a batch of look-ups past the last token stays in int32
    const cudaError_t e = pa::plan_decode_fp4(s->dtype, s->head_dim, s->num_heads / s->num_kv_heads, s->batch,
                                              s->num_kv_heads, s->block_size, (max_len + 31) / 32 + 1, plan);
    if (e == cudaErrorInvalidValue) {
        (void)cudaGetLastError();   // a too-large shared-memory request is not sticky; drop it
        return PA_ERR_UNSUPPORTED;
    }
    if (e != cudaSuccess) return PA_ERR_CUDA;
    return plan->grid > 0 ? PA_OK : PA_ERR_UNSUPPORTED;
}

// Records, group counters, then one counter per item.  Only the last part's
// size depends on the shape: a workspace serves every shape that it is large
// enough for.
struct WsLayout {
    size_t group_counters, counters, total;
};
WsLayout ws_of(const pa::Fp4Plan &plan) {
    WsLayout w;
    w.group_counters = (size_t)4 * plan.max_grid * pa::kFp4RecFloats * 4;
    w.counters = w.group_counters + (size_t)2 * plan.max_grid * 4;
    w.total = w.counters + (size_t)plan.items * 4;
    return w;
}

}  // namespace

extern "C" {

pa_status paged_kv_append_rope(const pa_shape *shape, const pa_rope *rope, const pa_new_rows *rows,
                               void *q_out, void *k_pool, void *v_pool,
                               const int32_t *block_table, const int32_t *positions,
                               const int32_t *counts, int32_t *err_word, pa_stream_t stream) {
    if (rope == nullptr) return PA_ERR_INVALID_ARG;
    return append(shape, rope, nullptr, rows, true, q_out, k_pool, v_pool, false, nullptr, 1.f, 1.f, block_table, positions,
                  counts, err_word, stream);
}

pa_status paged_kv_append_rope_axes(const pa_shape *shape, const pa_rope *rope, const pa_rope_axes *axes,
                                    const pa_new_rows *rows, void *q_out, void *k_pool, void *v_pool,
                                    const int32_t *block_table, const int32_t *positions,
                                    const int32_t *counts, int32_t *err_word, pa_stream_t stream) {
    if (rope == nullptr || axes == nullptr) return PA_ERR_INVALID_ARG;
    return append(shape, rope, axes, rows, true, q_out, k_pool, v_pool, false, nullptr, 1.f, 1.f, block_table, positions,
                  counts, err_word, stream);
}

pa_status paged_kv_append_fp4(const pa_shape *shape, const pa_new_rows *rows, uint8_t *k_pool,
                              uint8_t *v_pool, uint8_t *kv_scales, float k_scale, float v_scale,
                              const int32_t *block_table, const int32_t *positions,
                              const int32_t *counts, int32_t *err_word, pa_stream_t stream) {
    return append(shape, nullptr, nullptr, rows, false, nullptr, k_pool, v_pool, true, kv_scales, k_scale, v_scale,
                  block_table, positions, counts, err_word, stream);
}

pa_status paged_kv_append_rope_fp4(const pa_shape *shape, const pa_rope *rope,
                                   const pa_new_rows *rows, void *q_out, uint8_t *k_pool,
                                   uint8_t *v_pool, uint8_t *kv_scales, float k_scale,
                                   float v_scale, const int32_t *block_table,
                                   const int32_t *positions, const int32_t *counts,
                                   int32_t *err_word, pa_stream_t stream) {
    if (rope == nullptr) return PA_ERR_INVALID_ARG;
    return append(shape, rope, nullptr, rows, true, q_out, k_pool, v_pool, true, kv_scales, k_scale, v_scale, block_table,
                  positions, counts, err_word, stream);
}

pa_status paged_kv_gather_fp4(const pa_shape *shape, void *k_out, void *v_out, int32_t max_tokens,
                              const uint8_t *k_pool, const uint8_t *v_pool,
                              const uint8_t *kv_scales, float k_scale, float v_scale,
                              const int32_t *block_table, const int32_t *starts,
                              const int32_t *counts, int32_t *err_word, pa_stream_t stream) {
    pa_status st = check_fp4_shape(shape, false);
    if (st != PA_OK) return st;
    if (max_tokens < 0 || !factor_ok(k_scale) || !factor_ok(v_scale)) return PA_ERR_INVALID_ARG;
    if (shape->batch == 0 || max_tokens == 0) return PA_OK;
    if (k_out == nullptr || v_out == nullptr || k_pool == nullptr || v_pool == nullptr || kv_scales == nullptr ||
        block_table == nullptr || starts == nullptr)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(k_out) || !aligned16(v_out) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(kv_scales))
        return PA_ERR_MISALIGNED;
    pa::GatherFp4Params p{};
    p.k_out = k_out;
    p.v_out = v_out;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.scales = kv_scales;
    p.block_table = block_table;
    p.starts = starts;
    p.counts = counts;
    p.err_word = err_word;
    p.num_blocks = shape->num_blocks;
    p.block_stride_bytes = shape->block_stride;
    p.B = shape->batch;
    p.T = max_tokens;
    p.Hkv = shape->num_kv_heads;
    p.MB = shape->max_blocks_per_seq;
    p.bs = shape->block_size;
    p.bs_shift = log2_or_none(shape->block_size);
    p.k_g = k_scale;
    p.v_g = v_scale;
    return pa::launch_gather_fp4(shape->dtype, shape->head_dim, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

size_t paged_attention_fp4_workspace(const pa_shape *shape) {
    if (check_fp4_shape(shape, true) != PA_OK || shape->batch == 0) return 0;
    pa::Fp4Plan plan;
    if (plan_of(shape, &plan) != PA_OK) return 0;
    return ws_of(plan).total;
}

pa_status paged_attention_decode_fp4(const pa_shape *shape, void *out, const void *q,
                                     const uint8_t *k_pool, const uint8_t *v_pool,
                                     const uint8_t *kv_scales, float k_scale, float v_scale,
                                     const int32_t *block_table, const int32_t *seq_lens,
                                     float scale, int32_t window, void *workspace,
                                     size_t workspace_bytes, int32_t *err_word,
                                     pa_stream_t stream) {
    pa_status st = check_fp4_shape(shape, true);
    if (st != PA_OK) return st;
    if (window < 0 || !isfinite(scale) || !factor_ok(k_scale) || !factor_ok(v_scale)) return PA_ERR_INVALID_ARG;
    const float scale_log2 = (float)((double)scale * (double)k_scale * 1.4426950408889634);
    if (!isfinite(scale_log2)) return PA_ERR_INVALID_ARG;
    if (shape->batch == 0) return PA_OK;
    if (out == nullptr || q == nullptr || k_pool == nullptr || v_pool == nullptr || kv_scales == nullptr ||
        block_table == nullptr || seq_lens == nullptr || workspace == nullptr)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(kv_scales) ||
        !aligned16(workspace))
        return PA_ERR_MISALIGNED;
    pa::Fp4Plan plan;
    st = plan_of(shape, &plan);
    if (st != PA_OK) return st;
    const WsLayout w = ws_of(plan);
    if (workspace_bytes < w.total) return PA_ERR_WORKSPACE;
    pa::Fp4Decode f{};
    pa::DecodeParams &p = f.d;
    p.q = q;
    p.out = out;
    p.k_pool = reinterpret_cast<const char *>(k_pool);
    p.v_pool = reinterpret_cast<const char *>(v_pool);
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.err_word = err_word;
    p.num_blocks = shape->num_blocks;
    p.block_stride_bytes = shape->block_stride;
    p.B = shape->batch;
    p.H = shape->num_heads;
    p.Hkv = shape->num_kv_heads;
    p.D = shape->head_dim;
    p.MB = shape->max_blocks_per_seq;
    p.bs = shape->block_size;
    p.bs_shift = log2_or_none(shape->block_size);
    p.window = window;
    p.scale_log2 = scale_log2;
    char *ws = static_cast<char *>(workspace);
    p.records = reinterpret_cast<float *>(ws);
    p.group_counters = reinterpret_cast<int32_t *>(ws + w.group_counters);
    p.counters = reinterpret_cast<int32_t *>(ws + w.counters);
    p.rec_floats = pa::kFp4RecFloats;
    f.scales = kv_scales;
    f.v_g = v_scale;
    return pa::launch_decode_fp4(shape->dtype, f, plan, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // extern "C"
