// gather_fp4.cu -- rows of the 4-bit cache back as values.
//
// Bound by HBM: D/2 + D/16 bytes read and D elements written per row.  A
// thread turns one group of 16 codes (8 bytes) and its scale into 16 values
// (32 bytes of a 16-bit type); the groups of all heads of a token, K then V,
// are spread over the lanes of a warp, so that the output of a token is
// written in whole lines and the table is looked up once per token.
#include "fp4.cuh"
#include "pa_rope_fp4.h"

namespace pa {

constexpr int kGatherThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kGatherThreads) gather_fp4_kernel(const __grid_constant__ GatherFp4Params p) {
    grid_dependency_wait();
    allow_dependents();
    constexpr int G = D / 16;                      // groups per row
    const int b = blockIdx.x;
    const int n = p.counts != nullptr ? p.counts[b] : p.T;
    const int32_t start = p.starts[b];
    const bool reporter = threadIdx.x == 0 && blockIdx.y == 0;
    if (n < 0 || n > p.T) {
        if (reporter) report(p.err_word, PA_DEVERR_BAD_LEN);
        return;
    }
    const bool bad_pos = start < 0 || (int64_t)start + n > (int64_t)p.MB * p.bs;
    if (bad_pos && reporter) report(p.err_word, PA_DEVERR_BAD_POS);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_token = 2 * p.Hkv * G;
    const int per_warp = 32 / per_token > 1 ? 32 / per_token : 1;   // tokens of a warp side by side
    const int side = per_warp > 1 ? lane / per_token : 0;
    const int piece0 = per_warp > 1 ? lane - side * per_token : lane;
    const int step = (int)gridDim.y * (kGatherThreads / 32) * per_warp;
    for (int t0 = ((int)blockIdx.y * (kGatherThreads / 32) + warp) * per_warp; t0 < n; t0 += step) {
        const int t = t0 + side;
        if (t >= n || side >= per_warp) continue;
        const int32_t pos = start + t;
        int64_t blk = -1;
        int slot = 0;
        if (!bad_pos) {
            const int j = pos / p.bs;
            slot = pos - j * p.bs;
            blk = p.block_table[(int64_t)b * p.MB + j];
        }
        const bool ok = blk >= 0 && blk < p.num_blocks;
        if (!bad_pos && !ok && piece0 == 0) report(p.err_word, PA_DEVERR_BAD_BLOCK);
        const int64_t token = (int64_t)b * p.T + t;
        for (int i = piece0; i < per_token; i += per_warp > 1 ? per_token : 32) {
            const int gi = i % G;
            const int r = i / G;
            const bool is_v = r >= p.Hkv;
            const int h = is_v ? r - p.Hkv : r;
            float x[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = 0.f;
            if (ok) {
                const int64_t row = (int64_t)h * p.bs + slot;
                const uint2 w = __ldg(reinterpret_cast<const uint2 *>((is_v ? p.v_pool : p.k_pool) +
                                                                      blk * p.block_stride_bytes + row * (D / 2)) + gi);
                const uint32_t sc = __ldg(p.scales + ((blk * 2 + (is_v ? 1 : 0)) * p.Hkv * p.bs + row) * G + gi);
                const uint32_t s2 = e4m3x2_to_f16x2(sc | (sc << 8));
                const float g = is_v ? p.v_g : p.k_g;
                const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t f[4] = {e2m1x2_to_f16x2<0>(ww[k]), e2m1x2_to_f16x2<1>(ww[k]),
                                           e2m1x2_to_f16x2<2>(ww[k]), e2m1x2_to_f16x2<3>(ww[k])};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 v = f16x2_to_float2(hmul2_u32(f[j], s2));
                        x[8 * k + 2 * j] = v.x * g;
                        x[8 * k + 2 * j + 1] = v.y * g;
                    }
                }
            }
            T *dst = reinterpret_cast<T *>(is_v ? p.v_out : p.k_out) + (token * p.Hkv + h) * D + gi * 16;
            float lo[8], hi[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) lo[j] = x[j], hi[j] = x[8 + j];
            store8(dst, lo);
            store8(dst + 8, hi);
        }
    }
}

template <typename T, int D>
static cudaError_t launch_one(const GatherFp4Params &p, cudaStream_t stream) {
    const int per_token = 2 * p.Hkv * (D / 16);
    const int per_cta = (kGatherThreads / 32) * (32 / per_token > 1 ? 32 / per_token : 1);
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    int64_t gy = ((int64_t)p.T + per_cta - 1) / per_cta;
    const int64_t most = (32 * (int64_t)sms + p.B - 1) / p.B;   // about 32 CTAs per SM, then tokens in turn
    gy = gy > most ? most : gy;
    gy = gy > 65535 ? 65535 : gy;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.B, (unsigned)gy, 1);
    cfg.blockDim = dim3(kGatherThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = PA_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gather_fp4_kernel<T, D>, p);
}

template <typename T>
static cudaError_t launch_typed(int head_dim, const GatherFp4Params &p, cudaStream_t s) {
    switch (head_dim) {
        case 64: return launch_one<T, 64>(p, s);
        case 128: return launch_one<T, 128>(p, s);
        case 256: return launch_one<T, 256>(p, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_gather_fp4(int dtype, int head_dim, const GatherFp4Params &p, cudaStream_t stream) {
    if (p.B == 0 || p.T == 0) return cudaSuccess;
    switch (dtype) {
        case PA_F32: return launch_typed<float>(head_dim, p, stream);
        case PA_F16: return launch_typed<__half>(head_dim, p, stream);
        case PA_BF16: return launch_typed<__nv_bfloat16>(head_dim, p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pa
