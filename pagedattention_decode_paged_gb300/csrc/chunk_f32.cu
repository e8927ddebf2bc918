// chunk_f32.cu -- attention of several new tokens, fp32, on the CUDA cores.
//
// An item is 64 query rows (32 of each map in the differential form), tiles
// are 64 cache positions; 256 threads hold 4 x 4 scores each, then 4 rows of
// D/16 outputs (128 threads with 8 x 4 need fewer loads from shared memory, but
// then too few warps wait for them: 4 prompts of 1024 tokens, 16 heads on 4 of 128,
// 539 us for 490).  Products and sums are fp32 fused multiply-adds: the tensor
// cores' tf32 keeps 11 bits.  Two CTAs an SM, so that one computes while the
// other's tile is on its way.  35 TFLOP/s on those prompts, of 75 that the CUDA
// cores have: loads from shared memory (their pipe 71% busy) and waits for them, and at
// head_dim 128 the 128 registers that two CTAs leave a thread: it stores 84 to 88 bytes
// of its own and loads 308.
#include "chunk_sched.cuh"

namespace pa {

namespace {

using namespace chunk;

constexpr int kThreads = 256;
constexpr int kKT = 64;
constexpr int kRows = 64;

template <int D, bool DIFF>
struct Layout {
    static constexpr int E = DIFF ? D / 2 : D;
    static constexpr int kQPitch = E + 4, kPitch = D + 4, kPPitch = kKT + 4;   // floats: rows 4 banks apart
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kKV = kRows * kQPitch * 4;
    static constexpr uint32_t kK = kKV;                       // scores' tile, then the weights or rows of O
    static constexpr uint32_t kKBytes = kKT * (kPitch > kPPitch ? kPitch : kPPitch) * 4;
    static constexpr uint32_t kV = kK + kKBytes;
    static constexpr uint32_t kOff = kV + kKT * kPitch * 4;
    static constexpr uint32_t kSums = kOff + kKT * 8;
    static constexpr uint32_t kBad = kSums + kRows * 4;
    static constexpr uint32_t kPre = kBad + 16;
    static constexpr uint32_t kBytes = kPre + (kGroups + 1) * 8;
};

}  // namespace

template <int D, bool DIFF>
__global__ void __launch_bounds__(kThreads, 2) chunk_f32_kernel(const __grid_constant__ ChunkParams p) {
    using L = Layout<D, DIFF>;
    constexpr int E = L::E, R = DIFF ? kRows / 2 : kRows, NV = D / 16;
    grid_dependency_wait();
    allow_dependents();
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sb = smem_u32(smem);
    float *sq = reinterpret_cast<float *>(smem + L::kQ), *sk = reinterpret_cast<float *>(smem + L::kK);
    float *sv = reinterpret_cast<float *>(smem + L::kV), *sums = reinterpret_cast<float *>(smem + L::kSums);
    int64_t *off = reinterpret_cast<int64_t *>(smem + L::kOff);
    uint32_t *badm = reinterpret_cast<uint32_t *>(smem + L::kBad);
    int64_t *pre = reinterpret_cast<int64_t *>(smem + L::kPre);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, tx = tid & 15, ty = tid >> 4;

    Slices slices;
    Sched<R, kKT> it;
    int errors;
    const bool has = p.B <= kWarpSeqs ? it.locate(p, slices, &errors)
                                      : it.locate(p, slices, pre, Sched<R, kKT>::build(p, pre, tid, kThreads, 1, &errors));
    if (warp == 0) {
        if (p.B <= kWarpSeqs) errors = all_errors(p, errors);
        if (lane == 0) p.cuts[blockIdx.x] = cut_entry<R, kKT>(p, it, has, slices, errors);
    }
    if (!has) return;

    const int map = DIFF ? ty / 8 : 0;         // of this thread's rows 4 ty .. 4 ty + 3
    do {
        const Item x = it.x;
        const int n0 = x.i * R, nrows = min(R, x.cnt * p.G - n0);
        const int tmin = (int)by_group(p, n0), tmax = (int)by_group(p, n0 + nrows - 1);
        const int need_lo = p.window > 0 ? max(0, x.pos + tmin - p.window + 1) : 0, need_hi = x.pos + tmax;
        const int wlo_max = p.window > 0 ? max(0, x.pos + tmax - p.window + 1) : 0;
        for (int c = tid; c < kRows * (E / 4); c += kThreads) {
            const int row = c / (E / 4), ch = c % (E / 4), r = row % R, m = row / R, n = n0 + r;
            const float *src = reinterpret_cast<const float *>(p.q);
            if (r < nrows)
                src += ((int64_t)x.b * p.T + by_group(p, n)) * p.q_stride +
                       (int64_t)(x.hk * p.G + (n - (int)by_group(p, n) * p.G)) * D + m * E + ch * 4;
            cp16(sb + L::kQ + (row * L::kQPitch + ch * 4) * 4, src, r < nrows);
        }
        auto look_up = [&](int k) -> int64_t {     // place of row tid of tile k: -1 not needed, -2 bad
            const int t = (x.lo + k) * kKT + tid;
            if (tid >= kKT || k >= x.k1 || t < need_lo || t > need_hi) return -1;
            const int64_t o = row_offset(p, x.b, x.hk, t, D * 4);
            return o < 0 ? -2 : o;
        };
        int row_lo[4], row_hi[4];
        bool row_bad[4] = {false, false, false, false};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (ty * 4 + i) % R;
            const int pos = x.pos + (int)by_group(p, n0 + r);
            row_hi[i] = r < nrows ? pos : INT32_MAX;           // rows that are not there may see anything
            row_lo[i] = r < nrows && p.window > 0 ? max(0, pos - p.window + 1) : 0;
        }
        float o[4][NV], m[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j) o[i][j] = 0.f;
        }
        int64_t ahead = look_up(x.k0);
        for (int k = x.k0; k < x.k1; ++k) {
            if (tid < kKT) {
                off[tid] = ahead;
                const uint32_t b = __ballot_sync(0xffffffffu, ahead == -2);
                if (lane == 0) badm[warp] = b;
            }
            __syncthreads();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t dst = sb + (half ? L::kV : L::kK);
                const char *pool = half ? p.v_pool : p.k_pool;
                for (int c = tid; c < kKT * (D / 4); c += kThreads) {
                    const int row = c / (D / 4), ch = c % (D / 4);
                    const int64_t at = off[row];
                    cp16(dst + (row * L::kPitch + ch * 4) * 4, pool + (at < 0 ? 0 : at) + ch * 16, at >= 0);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
            ahead = look_up(k + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();
            // scores of rows 4 ty + i and positions tx + 16 j
            float s[4][4];
            {
                float2 e[4][4];                    // sums over even and odd d
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[i][j] = make_float2(0.f, 0.f);
                const float *q = sq + ty * 4 * L::kQPitch, *kk = sk + tx * L::kPitch + map * E;
#pragma unroll 2
                for (int d = 0; d < E; d += 4) {
                    float4 a[4], b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(q + i * L::kQPitch + d);
#pragma unroll
                    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(kk + j * 16 * L::kPitch + d);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            e[i][j] = fma2(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), e[i][j]);
                            e[i][j] = fma2(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), e[i][j]);
                        }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] = e[i][j].x + e[i][j].y;
            }
            const int t0 = (x.lo + k) * kKT;
            const bool partial = t0 < wlo_max || t0 + kKT - 1 > x.pos + tmin;
            const uint64_t bad = (uint64_t)badm[1] << 32 | badm[0];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mx = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = t0 + tx + 16 * j;
                    if (!(partial && (t < row_lo[i] || t > row_hi[i]))) mx = fmaxf(mx, s[i][j] * p.scale_log2);
                }
#pragma unroll
                for (int h = 1; h < 16; h <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, h));
                const float ref = mx == -INFINITY ? 0.f : mx, alpha = exp2f(m[i] - ref);
                m[i] = mx;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // the product unrounded: what the maximum was rounded to is the same for the whole row
                    const int t = t0 + tx + 16 * j;
                    const bool sees = !(partial && (t < row_lo[i] || t > row_hi[i]));
                    s[i][j] = sees ? exp2f(fmaf(s[i][j], p.scale_log2, -ref)) : 0.f;
                    sum += s[i][j];
                }
                l[i] = l[i] * alpha + sum;
#pragma unroll
                for (int j = 0; j < NV; ++j) o[i][j] *= alpha;
                if (bad != 0) {
                    const int a = max(0, row_lo[i] - t0), e = min(kKT - 1, row_hi[i] - t0);
                    if (a <= e && ((bad >> a) << a << (kKT - 1 - e)) != 0) row_bad[i] = true;
                }
            }
            __syncthreads();                       // all scores are there: the weights take the keys' place
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sk[(ty * 4 + i) * L::kPPitch + tx + 16 * j] = s[i][j];
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            // Where rows of the tile see different positions, a value that is not finite
            // must not reach the rows that do not see it, as 0 times it would.
            bool odd = false;
            if (partial)
                for (int c = tid; c < kKT * (D / 4); c += kThreads) {      // what this thread has copied
                    const uint4 v = *reinterpret_cast<const uint4 *>(sv + c / (D / 4) * L::kPitch + c % (D / 4) * 4);
                    odd |= (v.x & 0x7f800000u) == 0x7f800000u || (v.y & 0x7f800000u) == 0x7f800000u ||
                           (v.z & 0x7f800000u) == 0x7f800000u || (v.w & 0x7f800000u) == 0x7f800000u;
                }
            odd = __syncthreads_or(odd);
            const float *w = sk + ty * 4 * L::kPPitch;
            constexpr int V = NV >= 4 ? 4 : NV;    // neighbouring outputs: V tx + 16 V jj
            auto value = [&](int t, float (&v)[NV]) {
                const float *src = sv + t * L::kPitch + tx * V;
#pragma unroll
                for (int j = 0; j < NV; j += V) {
                    if constexpr (V == 4) *reinterpret_cast<float4 *>(v + j) = *reinterpret_cast<const float4 *>(src + j * 16);
                    else if constexpr (V == 2) *reinterpret_cast<float2 *>(v + j) = *reinterpret_cast<const float2 *>(src + j * 16);
                    else v[j] = src[j * 16];
                }
            };
            if (!odd) {
#pragma unroll 2
                for (int t = 0; t < kKT; t += 4) {
                    __align__(16) float a[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<float4 *>(a[i]) = *reinterpret_cast<const float4 *>(w + i * L::kPPitch + t);
#pragma unroll
                    for (int tt = 0; tt < 4; ++tt) {
                        __align__(16) float v[NV];
                        value(t + tt, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if constexpr (NV >= 2) {
#pragma unroll
                                for (int j = 0; j < NV; j += 2) {
                                    const float2 y = fma2(make_float2(a[i][tt], a[i][tt]), make_float2(v[j], v[j + 1]),
                                                          make_float2(o[i][j], o[i][j + 1]));
                                    o[i][j] = y.x;
                                    o[i][j + 1] = y.y;
                                }
                            } else {
                                o[i][0] = fmaf(a[i][tt], v[0], o[i][0]);
                            }
                        }
                    }
                }
            } else {
#pragma unroll 1
                for (int t = 0; t < kKT; ++t) {
                    __align__(16) float v[NV];
                    value(t, v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = w[i * L::kPPitch + t];
                        if (t0 + t >= row_lo[i] && t0 + t <= row_hi[i]) {
#pragma unroll
                            for (int j = 0; j < NV; ++j) o[i][j] = fmaf(a, v[j], o[i][j]);
                        }
                    }
                }
            }
            __syncthreads();
        }

        bool any_bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int h = 1; h < 16; h <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], h);
            if (row_bad[i]) l[i] = -1.f;
            any_bad |= row_bad[i] && (ty * 4 + i) % R < nrows;
        }
        if (any_bad && tx == 0) report(p.err_word, PA_DEVERR_BAD_BLOCK);
        const bool cut = it.cut();
        float *rec = p.records + ((int64_t)blockIdx.x * 2 + (x.k0 == 0)) * p.rec_floats;
        constexpr int V = NV >= 4 ? 4 : NV;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = ty * 4 + i;
            const float inv = cut ? 1.f : l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = tx * V + (j / V) * 16 * V + j % V;
                *(cut ? record_at(rec, kRows, row, c) : sk + row * L::kPitch + c) = o[i][j] * inv;
            }
            if (tx == 0) {
                if (cut) {
                    rec[kRows * D + row] = m[i];
                    rec[kRows * D + kRows + row] = l[i];
                } else {
                    sums[row] = l[i];
                }
            }
        }
        __syncthreads();
        if (!cut) {
            constexpr int N = D >= 32 ? D / 32 : 1;
            for (int r = warp; r < nrows; r += kThreads / 32) {
                const int n = n0 + r, e = D >= 32 ? lane * N : lane & (D - 1);
                finish_row<float, D, DIFF>(p, sk + r * L::kPitch + e, sk + (kRows / 2 + r) * L::kPitch + e,
                                           sums[r] < 0.f || (DIFF && sums[kRows / 2 + r] < 0.f),
                                           (int64_t)x.b * p.T + by_group(p, n), x.hk * p.G + n - (int)by_group(p, n) * p.G);
            }
            __syncthreads();
        }
    } while (it.next(p));
}

namespace {

template <int D, bool DIFF>
cudaError_t plan_one(ChunkPlan *plan) {
    static std::atomic<int> limit[64];
    static std::atomic<int64_t> cache[64];
    auto kern = chunk_f32_kernel<D, DIFF>;
    constexpr size_t smem = Layout<D, DIFF>::kBytes;
    cudaError_t e = ensure_smem_limit(kern, smem, limit);
    if (e != cudaSuccess) return e;
    int n = 0, sms = 0;
    e = resident_ctas(kern, kThreads, smem, cache, &n);
    if (e != cudaSuccess) return e;
    e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    if (n == 0) return cudaErrorInvalidValue;
    plan->grid = n * sms;
    plan->maps = DIFF ? 2 : 1;
    plan->rows = kRows / plan->maps;
    plan->rec_floats = chunk_rec_floats(kRows, D);
    return cudaSuccess;
}
template <int D, bool DIFF>
cudaError_t launch_one(const ChunkParams &p, const ChunkPlan &plan, cudaStream_t stream) {
    return launch_clustered(chunk_f32_kernel<D, DIFF>, plan.grid, kThreads, Layout<D, DIFF>::kBytes, 1, stream, p);
}

}  // namespace

cudaError_t plan_chunk_f32(int head_dim, bool diff, ChunkPlan *plan) {
    switch (head_dim) {
        case 16: return diff ? cudaErrorInvalidValue : plan_one<16, false>(plan);
        case 32: return diff ? plan_one<32, true>(plan) : plan_one<32, false>(plan);
        case 64: return diff ? plan_one<64, true>(plan) : plan_one<64, false>(plan);
        case 128: return diff ? plan_one<128, true>(plan) : plan_one<128, false>(plan);
    }
    return cudaErrorInvalidValue;
}
cudaError_t launch_chunk_f32(int head_dim, const ChunkParams &p, const ChunkPlan &plan, cudaStream_t stream) {
    const bool diff = plan.maps == 2;
    switch (head_dim) {
        case 16: return diff ? cudaErrorInvalidValue : launch_one<16, false>(p, plan, stream);
        case 32: return diff ? launch_one<32, true>(p, plan, stream) : launch_one<32, false>(p, plan, stream);
        case 64: return diff ? launch_one<64, true>(p, plan, stream) : launch_one<64, false>(p, plan, stream);
        case 128: return diff ? launch_one<128, true>(p, plan, stream) : launch_one<128, false>(p, plan, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pa
