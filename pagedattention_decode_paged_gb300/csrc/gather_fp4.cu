// gather_fp4.cu -- rows of the 4-bit cache back as values.
//
// Bound by HBM: D/2 + D/16 bytes read and D elements written per row, so mostly
// by writes.  A thread turns as many codes as make 16 bytes of output (8 of a
// 16-bit type, 4 of fp32), so that every store of a warp is 512 contiguous bytes
// (32 bytes a thread, stored as two halves, took 58.3 us where this takes 55.6 us:
// 32 contexts of 1500 to 2048 tokens, 8 heads of 128, bf16).  The pieces of all
// heads of a token, K then V, are spread over the lanes of a warp, which looks
// up the table once for the token.
#include "fp4.cuh"
#include "pa_rope_fp4.h"

namespace pa {

constexpr int kGatherThreads = 256;
constexpr int kGatherPieces = 8;   // pieces in flight per lane

template <typename T, int D>
__global__ void __launch_bounds__(kGatherThreads) gather_fp4_kernel(const __grid_constant__ GatherFp4Params p) {
    grid_dependency_wait();
    allow_dependents();
    constexpr int E = 16 / (int)sizeof(T), G = D / E;   // elements of a piece, pieces of a row
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
            const int j = p.bs_shift >= 0 ? pos >> p.bs_shift : pos / p.bs;
            slot = pos - j * p.bs;
            blk = __ldg(p.block_table + (int64_t)b * p.MB + j);
        }
        const bool ok = blk >= 0 && blk < p.num_blocks;
        if (!bad_pos && !ok && piece0 == 0) report(p.err_word, PA_DEVERR_BAD_BLOCK);
        const int64_t token = (int64_t)b * p.T + t;
        const int stride = per_warp > 1 ? per_token : 32;
#pragma unroll 1
        for (int i0 = piece0; i0 < per_token; i0 += kGatherPieces * stride) {
            uint32_t w[kGatherPieces], sc[kGatherPieces];
#pragma unroll
            for (int u = 0; u < kGatherPieces; ++u) {
                const int i = i0 + u * stride;
                w[u] = sc[u] = 0;
                if (ok && i < per_token) {
                    const int r = i / G, h = r < p.Hkv ? r : r - p.Hkv;
                    const int64_t row = (int64_t)h * p.bs + slot;
                    const uint8_t *codes = (r < p.Hkv ? p.k_pool : p.v_pool) + blk * p.block_stride_bytes + row * (D / 2) + i % G * (E / 2);
                    if constexpr (E == 8) w[u] = __ldg(reinterpret_cast<const uint32_t *>(codes));
                    else w[u] = __ldg(reinterpret_cast<const uint16_t *>(codes));
                    sc[u] = __ldg(p.scales + ((blk * 2 + (r < p.Hkv ? 0 : 1)) * p.Hkv * p.bs + row) * (D / 16) + i % G * E / 16);
                }
            }
#pragma unroll
            for (int u = 0; u < kGatherPieces; ++u) {
                const int i = i0 + u * stride;
                if (i >= per_token) break;
                const int r = i / G, h = r < p.Hkv ? r : r - p.Hkv;
                const float g = r < p.Hkv ? p.k_g : p.v_g;
                const uint32_t s2 = e4m3x2_to_f16x2(sc[u] | (sc[u] << 8));
                T *dst = reinterpret_cast<T *>(r < p.Hkv ? p.k_out : p.v_out) + (token * p.Hkv + h) * D + i % G * E;
                const float2 a = f16x2_to_float2(hmul2_u32(e2m1x2_to_f16x2<0>(w[u]), s2));
                const float2 c = f16x2_to_float2(hmul2_u32(e2m1x2_to_f16x2<1>(w[u]), s2));
                if constexpr (E == 8) {
                    const float2 d = f16x2_to_float2(hmul2_u32(e2m1x2_to_f16x2<2>(w[u]), s2));
                    const float2 e = f16x2_to_float2(hmul2_u32(e2m1x2_to_f16x2<3>(w[u]), s2));
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(Elem<T>::pack2(a.x * g, a.y * g), Elem<T>::pack2(c.x * g, c.y * g),
                                                                 Elem<T>::pack2(d.x * g, d.y * g), Elem<T>::pack2(e.x * g, e.y * g));
                } else {
                    *reinterpret_cast<float4 *>(dst) = make_float4(a.x * g, a.y * g, c.x * g, c.y * g);
                }
            }
        }
    }
}

template <typename T, int D>
static cudaError_t launch_one(const GatherFp4Params &p, cudaStream_t stream) {
    const int per_token = 2 * p.Hkv * (D * (int)sizeof(T) / 16);
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
