// chunk_merge.cu -- the second launch of attention of several new tokens: rows
// whose cache positions were cut between CTAs, joined from their records by
// the log-sum-exp identity (rescale each share's sum and weighted V by
// 2^(m_s - M) for the overall maximum M), as the split-KV reduce does.
//
// CTA (w, y) reads cuts[w]; where an item begins to be cut there, it joins rows
// 32 y to 32 y + 31 of it: lane r has row r, warp g a part of the columns, so
// that a record's rows are read in whole lines, each once; at most two records
// per CTA of the first launch exist, so the whole launch reads at most 2 * grid
// of them.  Few rows leave lanes over: those take the records in turn (1 token of 8
// heads behind 131071 of them, 38 records each: the call 123 us without, 104 so).
// The joined rows go through shared memory to a warp each.  Bound by latency: cuts,
// records and outputs are three dependent trips to L2 (4 tokens behind 2048 in 32
// sequences, 64 heads: 5 MB of records, about 4 us after the first launch, 8.9 alone).
#include "chunk_sched.cuh"

namespace pa {

namespace {

constexpr int kMergeThreads = 256;
constexpr int kMergeRows = 32;

// Zeros in the rows of the sequences whose positions are out of range, by all threads
// of the launch (a prompt of 16384 tokens, 64 heads of 128, is 268 MB).
__device__ __noinline__ void zero_bad_sequences(const ChunkParams &p, int row_bytes) {
    const int64_t threads = (int64_t)gridDim.x * gridDim.y * kMergeThreads;
    const int64_t me = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kMergeThreads + threadIdx.x;
    for (int b = 0; b < p.B; ++b) {
        int pos, error;
        chunk::seq_of(p, b, &pos, &error);
        if (error != PA_DEVERR_BAD_POS) continue;
        const int64_t token = (int64_t)p.H * row_bytes / 16;
        const int64_t n = (p.counts != nullptr ? __ldg(p.counts + b) : p.T) * token;
        uint4 *out = reinterpret_cast<uint4 *>(p.out) + (int64_t)b * p.T * token;
        for (int64_t i = me; i < n; i += threads) out[i] = make_uint4(0, 0, 0, 0);
    }
}

// rows: of a map in a record.
template <typename T, int D, bool DIFF>
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const __grid_constant__ ChunkParams p, const int rows) {
    grid_dependency_wait();
    allow_dependents();
    constexpr int MAPS = DIFF ? 2 : 1;
    constexpr int WARPS = kMergeThreads / 32, PARTS = D / 4 < WARPS ? D / 4 : WARPS, C4 = D / 4 / PARTS;   // float4 of a thread
    __shared__ float joined[kMergeRows][D + 4];
    __shared__ int zero[kMergeRows];
    const int w = blockIdx.x;
    const ChunkCut cut = p.cuts[w];
    const int r0 = blockIdx.y * kMergeRows;
    if (cut.zeros != 0) zero_bad_sequences(p, D * (int)sizeof(T));
    if (cut.b < 0 || r0 >= cut.rows) return;
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    // A state of each CTA that shares the item.  The launch before writes them while this
    // one may be resident already, so they are not for the read-only path.
    const int states = cut.last - w + 2, all = rows * MAPS;
    auto record = [&](int s) { return p.records + (int64_t)(s == 0 ? (w - 1) * 2 + 1 : (w - 1 + s) * 2) * p.rec_floats; };
    // rows of a warp: 8, 16 or 32; lanes `take` and on of a row take every `step`th state
    const int left = cut.rows - r0, lrows = left <= 8 ? 8 : left <= 16 ? 16 : 32, step = 32 / lrows, take = lane / lrows;
    const int i_row = lane & (lrows - 1);
    const int r = r0 + min(i_row, left - 1);
    bool bad = false;
    if (part < PARTS) {
#pragma unroll 1
        for (int map = 0; map < MAPS; ++map) {
            const int row = map * rows + r;
            float M = -INFINITY;
#pragma unroll 8
            for (int s = take; s < states; s += step) {
                const float *ml = record(s) + (int64_t)all * D + row;
                M = fmaxf(M, __ldcg(ml));
                bad |= __ldcg(ml + all) < 0.f;
            }
            for (int h = lrows; h < 32; h <<= 1) {
                M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, h));
                bad |= __shfl_xor_sync(0xffffffffu, (int)bad, h) != 0;
            }
            float L = 0.f;
            float4 acc[C4];
#pragma unroll
            for (int i = 0; i < C4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int s = take; s < states; s += step) {
                const float *rec = record(s), *ml = rec + (int64_t)all * D + row;
                const float f = merge_weight(__ldcg(ml), M);
                L += f * __ldcg(ml + all);
#pragma unroll
                for (int i = 0; i < C4; ++i) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(rec) + (part * C4 + i) * all + row);
                    acc[i].x += f * v.x, acc[i].y += f * v.y, acc[i].z += f * v.z, acc[i].w += f * v.w;
                }
            }
            for (int h = lrows; h < 32; h <<= 1) {
                L += __shfl_xor_sync(0xffffffffu, L, h);
#pragma unroll
                for (int i = 0; i < C4; ++i) {
                    acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, h);
                    acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, h);
                    acc[i].z += __shfl_xor_sync(0xffffffffu, acc[i].z, h);
                    acc[i].w += __shfl_xor_sync(0xffffffffu, acc[i].w, h);
                }
            }
            float inv = L == 0.f ? 0.f : 1.f / L;
            if (map == 1) {                        // o_1 - lambda o_2
                const uint32_t n = cut.n0 + r;
                inv *= -__ldg(p.lambdas + cut.hk * p.G + (int)(n - chunk::by_group(p, n) * p.G));
            }
            if (take != 0) continue;
#pragma unroll
            for (int i = 0; i < C4; ++i) {
                float4 &y = *reinterpret_cast<float4 *>(&joined[i_row][(part * C4 + i) * 4]);
                const float4 before = map == 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : y;
                y = make_float4(fmaf(acc[i].x, inv, before.x), fmaf(acc[i].y, inv, before.y), fmaf(acc[i].z, inv, before.z),
                                fmaf(acc[i].w, inv, before.w));
            }
        }
        if (part == 0 && take == 0) zero[i_row] = bad;
    }
    __syncthreads();
    constexpr int N = D >= 32 ? D / 32 : 1;
    const int at = D >= 32 ? lane * N : lane & (D - 1);
    for (int i = part; i < min(kMergeRows, cut.rows - r0); i += WARPS) {
        const uint32_t n = cut.n0 + r0 + i, t = chunk::by_group(p, n);
        chunk::finish_row<T, D, DIFF>(p, &joined[i][at], nullptr, zero[i] != 0, (int64_t)cut.b * p.T + t,
                                      cut.hk * p.G + (int)(n - t * p.G));
    }
}

template <typename T, int D>
cudaError_t launch_typed(const ChunkParams &p, const ChunkPlan &plan, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)plan.grid, (unsigned)((plan.rows + kMergeRows - 1) / kMergeRows), 1);
    cfg.blockDim = dim3(kMergeThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = PA_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (plan.maps == 2) return cudaLaunchKernelEx(&cfg, chunk_merge_kernel<T, D, true>, p, plan.rows);
    return cudaLaunchKernelEx(&cfg, chunk_merge_kernel<T, D, false>, p, plan.rows);
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
