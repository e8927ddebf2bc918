// chunk_merge.cu -- the second launch of attention of several new tokens: rows
// whose cache positions were cut between CTAs, joined from their records by
// the log-sum-exp identity (rescale each share's sum and weighted V by
// 2^(m_s - M) for the overall maximum M), as the split-KV reduce does.
//
// CTA (w, y) reads cuts[w]; where an item begins to be cut there, its rows are
// spread over the warps of the y.  A row's records are read once, 128 bytes
// and more at a time; at most two records per CTA of the first launch exist,
// so the whole launch reads at most 2 * grid of them.
#include "chunk_sched.cuh"

namespace pa {

namespace {

constexpr int kMergeThreads = 256;
constexpr int kMergeY = 8;

template <typename T, int D, bool DIFF>
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const __grid_constant__ ChunkParams p, const int rows, const int fold) {
    grid_dependency_wait();
    allow_dependents();
    constexpr int N = D >= 32 ? D / 32 : 1, MAPS = DIFF ? 2 : 1;
    const int w = blockIdx.x;
    const int4 c = p.cuts[w];
    if (c.x < 0) return;
    const int lane = threadIdx.x & 31;
    const int ctas = c.w - w + 2;
    const int cnt = p.counts != nullptr ? __ldg(p.counts + c.x) : p.T;
    const int n0 = c.z * rows, valid = min(rows, cnt * p.G - n0);
    // states of a row: one of each CTA, or two (a short item's rows r and fold + r)
    const bool two = valid <= fold;
    const int sharers = two ? 2 * ctas : ctas;
    auto record = [&](int s) {
        const int cta = two ? s >> 1 : s;
        return p.records + ((int64_t)(cta == 0 ? (w - 1) * 2 + 1 : (w - 1 + cta) * 2)) * p.rec_floats;
    };
    auto row_of = [&](int s, int row) { return two && (s & 1) ? fold + row : row; };
    for (int r = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5); r < valid; r += kMergeY * (kMergeThreads / 32)) {
        float o[MAPS][N];
        bool bad = false;
#pragma unroll
        for (int map = 0; map < MAPS; ++map) {
            const int row = map * rows + r;
            // lane s has the weight of share s, 32 shares at a time
            float M = -INFINITY;
            for (int s = lane; s < sharers; s += 32) {
                const float *ml = record(s) + (int64_t)rows * MAPS * D + row_of(s, row);
                M = fmaxf(M, __ldg(ml));
                bad |= __ldg(ml + rows * MAPS) < 0.f;
            }
            M = warp_max_f32(M);
            bad = __any_sync(0xffffffffu, bad);
            float L = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) o[map][i] = 0.f;
            for (int s0 = 0; s0 < sharers; s0 += 32) {
                float f = 0.f;
                if (s0 + lane < sharers) {
                    const float *ml = record(s0 + lane) + (int64_t)rows * MAPS * D + row_of(s0 + lane, row);
                    f = merge_weight(__ldg(ml), M);
                    L += f * __ldg(ml + rows * MAPS);
                }
                const int here = min(32, sharers - s0);
                // 8 shares' values on their way at once
                for (int s1 = 0; s1 < here; s1 += 8) {
                    float a[8][N];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int s = s0 + min(s1 + j, here - 1);
                        const float *src = record(s) + (int64_t)row_of(s, row) * D + lane * N;
                        if (D >= 32 || lane < D) {
                            if constexpr (N % 4 == 0) {
#pragma unroll
                                for (int i = 0; i < N; i += 4)
                                    *reinterpret_cast<float4 *>(a[j] + i) = __ldg(reinterpret_cast<const float4 *>(src + i));
                            } else {
#pragma unroll
                                for (int i = 0; i < N; ++i) a[j][i] = __ldg(src + i);
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float fj = __shfl_sync(0xffffffffu, f, min(s1 + j, 31));
                        if (s1 + j < here)
#pragma unroll
                            for (int i = 0; i < N; ++i) o[map][i] += fj * a[j][i];
                    }
                }
            }
#pragma unroll
            for (int h = 16; h > 0; h >>= 1) L += __shfl_xor_sync(0xffffffffu, L, h);
            const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
            for (int i = 0; i < N; ++i) o[map][i] *= inv;
        }
        const int n = n0 + r;
        chunk::finish_row<T, D, DIFF>(p, o[0], o[MAPS - 1], bad, (int64_t)c.x * p.T + n / p.G, c.y * p.G + n % p.G);
    }
}

template <typename T, int D>
cudaError_t launch_typed(const ChunkParams &p, const ChunkPlan &plan, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)plan.grid, kMergeY, 1);
    cfg.blockDim = dim3(kMergeThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = PA_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (plan.maps == 2) return cudaLaunchKernelEx(&cfg, chunk_merge_kernel<T, D, true>, p, plan.rows, plan.fold);
    return cudaLaunchKernelEx(&cfg, chunk_merge_kernel<T, D, false>, p, plan.rows, plan.fold);
}

}  // namespace

cudaError_t launch_chunk_merge(int dtype, int head_dim, const ChunkParams &p, const ChunkPlan &plan, cudaStream_t stream) {
    if (dtype == PA_F32) {
        switch (head_dim) {
            case 16: return launch_typed<float, 16>(p, plan, stream);
            case 32: return launch_typed<float, 32>(p, plan, stream);
            case 64: return launch_typed<float, 64>(p, plan, stream);
            case 128: return launch_typed<float, 128>(p, plan, stream);
        }
        return cudaErrorInvalidValue;
    }
    if (dtype == PA_F16) {
        switch (head_dim) {
            case 32: return launch_typed<__half, 32>(p, plan, stream);
            case 64: return launch_typed<__half, 64>(p, plan, stream);
            case 128: return launch_typed<__half, 128>(p, plan, stream);
            case 256: return launch_typed<__half, 256>(p, plan, stream);
        }
        return cudaErrorInvalidValue;
    }
    switch (head_dim) {
        case 32: return launch_typed<__nv_bfloat16, 32>(p, plan, stream);
        case 64: return launch_typed<__nv_bfloat16, 64>(p, plan, stream);
        case 128: return launch_typed<__nv_bfloat16, 128>(p, plan, stream);
        case 256: return launch_typed<__nv_bfloat16, 256>(p, plan, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pa
