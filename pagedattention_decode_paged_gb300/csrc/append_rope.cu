// append_rope.cu -- per-head norm, position rotation and append in one pass,
// into a cache of the new rows' type or into the 4-bit cache.
//
// Where a row goes follows "KV Cache and BlockManager" (dpshk.com/news/5906718)
// s4.4 and the valid-length rule of "A strange KV Cache bug"
// (dpshk.com/news/5937191) s2.4, as append.cu; the norm, the rotation and the
// 4-bit scheme are not on the pages (include/pagedattn_rope.h,
// include/pagedattn_fp4.h state them).
//
// Every element is read once and written once, so the kernel is bound by HBM
// for prompts and by launch and the dependent loads (position, table entry and
// cosines, rows) for single tokens.  D/8 lanes hold a row, 8 elements each:
// 16 bytes of a 16-bit type, so a warp moves whole 128-byte lines.  The mean
// square is a shuffle sum over those lanes; a rotation pair (i, i + R/2) lies
// R/16 lanes apart and is one shuffle per element, a pair (2i, 2i + 1) lies
// in one lane.  A thread keeps its cosines and sines for all the heads of a
// token that it visits.  The rotation is written with separately rounded
// products and sums: a few more instructions than fused ones, hidden behind
// the loads, and the 4-bit codes then are those of the stated formula.
#include "fp4.cuh"
#include "pa_rope_fp4.h"

namespace pa {

constexpr int kRopeThreads = 256;

// The row's 8 elements of this lane as 4-bit codes into `dst` (4 bytes) and
// the group's scale into `sdst`: a group of 16 is two neighbouring lanes.
// All lanes of the warp call; `write` says whose row goes to the cache.
__device__ __forceinline__ void store_fp4(const float (&x)[8], float g, bool write, uint32_t *dst, uint8_t *sdst,
                                          bool first_of_group) {
    float a = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(x[j]));   // a NaN loses against a number
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    const uint32_t code = f32_to_e4m3(__fdiv_rn(a, __fmul_rn(6.f, g)));
    const float t = __fmul_rn(f16x2_to_float2(e4m3x2_to_f16x2(code)).x, g);
    if (!write) return;
    uint32_t w = 0;
    if (t > 0.f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo = __fdiv_rn(x[2 * j], t), hi = __fdiv_rn(x[2 * j + 1], t);
            lo = lo == lo ? lo : 0.f;
            hi = hi == hi ? hi : 0.f;
            w |= f32x2_to_e2m1x2(lo, hi) << (8 * j);
        }
    }
    *dst = w;
    if (first_of_group) *sdst = (uint8_t)code;
}

// grid: x = sequence, y = stripe of tokens, z = stripe of rows of a token.
template <typename T, int D, bool FP4>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeAppendParams p) {
    grid_dependency_wait();
    allow_dependents();
    constexpr int LPR = D / 8;                     // lanes per row
    constexpr int RPB = kRopeThreads / LPR;        // rows per pass
    const int b = blockIdx.x;
    const int n = p.counts != nullptr ? p.counts[b] : p.T;
    const int32_t start = p.positions[b];
    const bool reporter = threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
    if (n < 0 || n > p.T) {
        if (reporter) report(p.err_word, PA_DEVERR_BAD_LEN);
        return;
    }
    const bool bad_pos = start < 0 || (int64_t)start + n > (int64_t)p.MB * p.bs ||
                         (p.R > 0 && (int64_t)start + n > (int64_t)p.max_position);
    if (bad_pos && reporter) report(p.err_word, PA_DEVERR_BAD_POS);

    const int HQ = p.q != nullptr ? p.H : 0;
    const int rows = HQ + 2 * p.Hkv;               // of a token
    const int per_pass = RPB / rows > 1 ? RPB / rows : 1;   // tokens side by side when rows are few
    const int lr = threadIdx.x / LPR, sub = threadIdx.x % LPR, d0 = sub * 8;
    const int side = per_pass > 1 ? lr / rows : 0;
    const int first_row = per_pass > 1 ? lr - side * rows : lr + (int)blockIdx.z * RPB;
    const int row_step = per_pass > 1 ? rows : RPB * (int)gridDim.z;
    const bool lane_rot = d0 < p.R;
    const int half = p.R / 16;                     // lanes between the two elements of a pair
    const int partner = !p.pairs && lane_rot ? (int)(threadIdx.x & 31) + (sub < half ? half : -half) : (int)(threadIdx.x & 31);

    for (int t0 = (int)blockIdx.y * per_pass; t0 < n; t0 += (int)gridDim.y * per_pass) {
        const int t = t0 + side;
        const bool live = t < n && side < per_pass;
        const int32_t pos = start + t;
        const int64_t token = (int64_t)b * p.T + t;
        int64_t blk = -1;
        int slot = 0;
        float c[8], s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = 1.f, s[j] = 0.f;
        if (live && !bad_pos) {
            const int j = pos / p.bs;
            slot = pos - j * p.bs;
            blk = p.block_table[(int64_t)b * p.MB + j];
            if (lane_rot) {
                const float *cs = p.cos_sin + (int64_t)pos * p.R;
                if (p.pairs) {
                    const float4 c4 = *reinterpret_cast<const float4 *>(cs + d0 / 2);
                    const float4 s4 = *reinterpret_cast<const float4 *>(cs + p.R / 2 + d0 / 2);
                    c[0] = c[1] = c4.x, c[2] = c[3] = c4.y, c[4] = c[5] = c4.z, c[6] = c[7] = c4.w;
                    s[0] = -s4.x, s[1] = s4.x, s[2] = -s4.y, s[3] = s4.y;
                    s[4] = -s4.z, s[5] = s4.z, s[6] = -s4.w, s[7] = s4.w;
                } else {
                    const int i = sub < half ? d0 : d0 - p.R / 2;
                    load8(cs + i, c);
                    load8(cs + p.R / 2 + i, s);
                    if (sub < half)
#pragma unroll
                        for (int k = 0; k < 8; ++k) s[k] = -s[k];
                }
            }
        }
        const bool to_cache = blk >= 0 && blk < p.num_blocks;
        if (live && !bad_pos && !to_cache && first_row == 0 && sub == 0) report(p.err_word, PA_DEVERR_BAD_BLOCK);

        // whole warps stay together: the shuffles below need every lane
        for (int r = first_row; __any_sync(0xffffffffu, live && r < rows); r += row_step) {
            const bool mine = live && r < rows;
            const bool is_q = r < HQ, is_v = r >= HQ + p.Hkv;
            const int h = is_q ? r : (is_v ? r - HQ - p.Hkv : r - HQ);
            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (mine && !bad_pos) {
                const T *src = is_q   ? reinterpret_cast<const T *>(p.q) + token * p.q_stride
                               : is_v ? reinterpret_cast<const T *>(p.v) + token * p.v_stride
                                      : reinterpret_cast<const T *>(p.k) + token * p.k_stride;
                load8(src + (int64_t)h * D + d0, x);
            }
            const T *w = reinterpret_cast<const T *>(is_q ? p.q_weight : p.k_weight);
            if (p.q_weight != nullptr || p.k_weight != nullptr) {
                float sq = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sq = fmaf(x[j], x[j], sq);
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
                if (!is_v && w != nullptr && mine && !bad_pos) {
                    const float rstd = __frsqrt_rn(__fadd_rn(sq * (1.f / D), p.eps));
                    float wf[8];
                    load8(w + d0, wf);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(__fmul_rn(x[j], rstd), wf[j]);
                }
            }
            if (p.R > 0) {
                float y[8];
                if (p.pairs) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], partner);
                }
                if (lane_rot && !is_v)
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(__fmul_rn(x[j], c[j]), __fmul_rn(y[j], s[j]));
            }
            if (mine && is_q) store8(reinterpret_cast<T *>(p.q_out) + (token * p.H + h) * D + d0, x);
            const int64_t row = (int64_t)h * p.bs + slot;
            char *pool = (is_v ? p.v_pool : p.k_pool) + blk * p.block_stride_bytes;
            const bool write = mine && !is_q && to_cache;
            if constexpr (FP4) {
                uint8_t *sd = p.scales + ((blk * 2 + (is_v ? 1 : 0)) * p.Hkv * p.bs + row) * (D / 16) + sub / 2;
                store_fp4(x, is_v ? p.v_g : p.k_g, write, reinterpret_cast<uint32_t *>(pool + row * (D / 2)) + sub, sd,
                          (sub & 1) == 0);
            } else {
                if (write) store8(reinterpret_cast<T *>(pool) + row * D + d0, x);
            }
        }
    }
}

template <typename T, int D, bool FP4>
static cudaError_t launch_one(const RopeAppendParams &p, cudaStream_t stream) {
    constexpr int RPB = kRopeThreads / (D / 8);
    const int rows = (p.q != nullptr ? p.H : 0) + 2 * p.Hkv;
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int per_pass = RPB / rows > 1 ? RPB / rows : 1;
    int64_t gy = ((int64_t)p.T + per_pass - 1) / per_pass;
    gy = gy > 65535 ? 65535 : gy;
    // few tokens: a token's rows over several CTAs, until every SM has one
    const int passes = (rows + RPB - 1) / RPB;
    int64_t gz = 2 * (int64_t)sms / ((int64_t)p.B * gy);
    gz = gz < 1 ? 1 : (gz > passes ? passes : gz);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.B, (unsigned)gy, (unsigned)gz);
    cfg.blockDim = dim3(kRopeThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = PA_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_append_kernel<T, D, FP4>, p);
}

bool rope_append_supported(int dtype, int head_dim, bool fp4) {
    if (fp4) return fp4_head_dim(head_dim);
    if (dtype == PA_F32) return head_dim == 16 || head_dim == 32 || head_dim == 64 || head_dim == 128;
    return head_dim == 32 || head_dim == 64 || head_dim == 128 || head_dim == 256;
}

template <typename T>
static cudaError_t launch_typed(int head_dim, bool fp4, const RopeAppendParams &p, cudaStream_t s) {
    if (fp4) {
        switch (head_dim) {
            case 64: return launch_one<T, 64, true>(p, s);
            case 128: return launch_one<T, 128, true>(p, s);
            case 256: return launch_one<T, 256, true>(p, s);
        }
        return cudaErrorInvalidValue;
    }
    switch (head_dim) {
        case 16:
            if constexpr (sizeof(T) == 4) return launch_one<T, 16, false>(p, s);
            break;
        case 32: return launch_one<T, 32, false>(p, s);
        case 64: return launch_one<T, 64, false>(p, s);
        case 128: return launch_one<T, 128, false>(p, s);
        case 256:
            if constexpr (sizeof(T) == 2) return launch_one<T, 256, false>(p, s);
            break;
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_rope_append(int dtype, int head_dim, bool fp4, const RopeAppendParams &p, cudaStream_t stream) {
    if (p.B == 0 || p.T == 0) return cudaSuccess;
    switch (dtype) {
        case PA_F32: return launch_typed<float>(head_dim, fp4, p, stream);
        case PA_F16: return launch_typed<__half>(head_dim, fp4, p, stream);
        case PA_BF16: return launch_typed<__nv_bfloat16>(head_dim, fp4, p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pa
