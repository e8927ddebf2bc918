// gather_fp4.cu -- rows of the 4-bit cache back as values.
//
// Bound by HBM: D/2 + D/16 bytes read and D elements written per row.  A lane
// turns as many codes as make 16 bytes of output (8 of a 16-bit type, 4 of
// fp32), so that every store of a warp is 512 contiguous bytes, and a warp looks
// up the table once for a token, whose rows of keys and values it then walks by
// constant steps: 46 us for 32 contexts of 1500 to 2048 tokens, 8 heads of 128,
// bf16 (222 MB written, 62 MB read; 6.2 TB/s).  With the place of every 16 bytes
// worked out by itself the same stores took 55.6 us, 120 instructions each, and
// 32 bytes a lane, stored as two halves, 58.3 us.
#include "fp4.cuh"
#include "pa_rope_fp4.h"

namespace pa {

constexpr int kGatherThreads = 128;   // 256: prompts of 366 to 1023 tokens 7.1 us, 6.8 so; 64: 7.3
constexpr int kGatherRows = 4;     // pieces of K, and of V, in flight per lane

template <typename T, int D>
struct GatherCfg {
    static constexpr int E = 16 / (int)sizeof(T), G = D / E;   // elements of a piece, pieces of a row
    static constexpr int LPR = G < 32 ? G : 32;                // lanes of a row, each with G / LPR of its pieces
    static constexpr int RPW = 32 / LPR;                       // rows a warp takes side by side
};

// 16 bytes of output: the codes w, under the scale byte sc, times g.
template <typename T>
__device__ __forceinline__ void put_values(T *dst, uint32_t w, uint32_t sc, float g) {
    const uint32_t s2 = e4m3x2_to_f16x2(sc * 0x101u);
    const float2 a = f16x2_to_float2(hmul2_u32(e2m1x2_to_f16x2<0>(w), s2));
    const float2 c = f16x2_to_float2(hmul2_u32(e2m1x2_to_f16x2<1>(w), s2));
    if constexpr (sizeof(T) == 2) {
        const float2 d = f16x2_to_float2(hmul2_u32(e2m1x2_to_f16x2<2>(w), s2));
        const float2 e = f16x2_to_float2(hmul2_u32(e2m1x2_to_f16x2<3>(w), s2));
        *reinterpret_cast<uint4 *>(dst) = make_uint4(Elem<T>::pack2(a.x * g, a.y * g), Elem<T>::pack2(c.x * g, c.y * g),
                                                     Elem<T>::pack2(d.x * g, d.y * g), Elem<T>::pack2(e.x * g, e.y * g));
    } else {
        *reinterpret_cast<float4 *>(dst) = make_float4(a.x * g, a.y * g, c.x * g, c.y * g);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kGatherThreads) gather_fp4_kernel(const __grid_constant__ GatherFp4Params p) {
    grid_dependency_wait();
    allow_dependents();
    using C = GatherCfg<T, D>;
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
    // few heads: the rows side by side are those of several tokens
    const int tokens = p.Hkv < C::RPW ? C::RPW / p.Hkv : 1, rows = tokens > 1 ? p.Hkv : C::RPW;
    const int side = lane / C::LPR / rows, h0 = lane / C::LPR - side * rows, c0 = lane % C::LPR;
    const int64_t code_step = (int64_t)C::RPW * p.bs * (D / 2), scale_step = (int64_t)C::RPW * p.bs * (D / 16);
    const int64_t v_codes = (int64_t)(reinterpret_cast<uintptr_t>(p.v_pool) - reinterpret_cast<uintptr_t>(p.k_pool));
    const int64_t v_scales = (int64_t)p.Hkv * p.bs * (D / 16);
    T *const k_out = reinterpret_cast<T *>(p.k_out), *const v_out = reinterpret_cast<T *>(p.v_out);
    const int64_t step = (int64_t)gridDim.y * (kGatherThreads / 32) * tokens;
    for (int64_t t = ((int64_t)blockIdx.y * (kGatherThreads / 32) + warp) * tokens + side; t < n && side < tokens; t += step) {
        const int32_t pos = start + (int32_t)t;
        int64_t blk = -1;
        int slot = 0;
        if (!bad_pos) {
            const int j = p.bs_shift >= 0 ? pos >> p.bs_shift : pos / p.bs;
            slot = pos - j * p.bs;
            blk = __ldg(p.block_table + (int64_t)b * p.MB + j);
        }
        const bool ok = blk >= 0 && blk < p.num_blocks;
        if (!bad_pos && !ok && h0 == 0 && c0 == 0) report(p.err_word, PA_DEVERR_BAD_BLOCK);
        const int64_t row = (int64_t)h0 * p.bs + slot;
        const uint8_t *cd = p.k_pool + blk * p.block_stride_bytes + row * (D / 2) + c0 * (C::E / 2);
        const uint8_t *sd = p.scales + (blk * 2 * p.Hkv * p.bs + row) * (D / 16) + c0 * C::E / 16;
        int64_t dst = (((int64_t)b * p.T + t) * p.Hkv + h0) * D + c0 * C::E;
#pragma unroll 1
        for (int h = h0; h < p.Hkv; h += kGatherRows * C::RPW) {
#pragma unroll
            for (int cj = 0; cj < C::G / C::LPR; ++cj) {
                constexpr int kCol = 32 * C::E;        // elements to a lane's next piece of a row
                uint32_t w[2][kGatherRows], sc[2][kGatherRows];
#pragma unroll
                for (int u = 0; u < kGatherRows; ++u) {
                    const uint8_t *cu = cd + u * code_step + cj * (kCol / 2), *su = sd + u * scale_step + cj * (kCol / 16);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        w[kv][u] = sc[kv][u] = 0;
                        if (ok && h + u * C::RPW < p.Hkv) {
                            const uint8_t *codes = cu + (kv ? v_codes : 0);
                            if constexpr (C::E == 8) w[kv][u] = __ldg(reinterpret_cast<const uint32_t *>(codes));
                            else w[kv][u] = __ldg(reinterpret_cast<const uint16_t *>(codes));
                            sc[kv][u] = __ldg(su + (kv ? v_scales : 0));
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < kGatherRows; ++u) {
                    if (h + u * C::RPW >= p.Hkv) break;
                    const int64_t at = dst + u * (C::RPW * D) + cj * kCol;
                    put_values<T>(k_out + at, w[0][u], sc[0][u], p.k_g);
                    put_values<T>(v_out + at, w[1][u], sc[1][u], p.v_g);
                }
            }
            cd += kGatherRows * code_step;
            sd += kGatherRows * scale_step;
            dst += kGatherRows * C::RPW * D;
        }
    }
}

template <typename T, int D>
static cudaError_t launch_one(const GatherFp4Params &p, cudaStream_t stream) {
    const int per_cta = (kGatherThreads / 32) * (p.Hkv < GatherCfg<T, D>::RPW ? GatherCfg<T, D>::RPW / p.Hkv : 1);
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    int64_t gy = ((int64_t)p.T + per_cta - 1) / per_cta;
    // about 256 warps per SM, then tokens in turn (64 warps: 50.5 us for the 32 contexts,
    // 46.0 so, 46.6 at 1024)
    const int64_t most = (64 * (int64_t)sms + p.B - 1) / p.B;
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
