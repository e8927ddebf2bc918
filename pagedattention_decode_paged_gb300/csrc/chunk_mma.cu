// chunk_mma.cu -- attention of several new tokens, 16-bit types, on the
// warp-level tensor-core instructions (mma.sync m16n8k16): every head_dim and
// every block size.
//
// An item is 64 query rows (32 of each map in the differential form), a warp
// 16 of them; tiles are 64 cache positions.  Per tile
//     S = Q K^T,  P = 2^(scale log2(e) S - m),  O = O 2^(m_old - m) + P V
// with the running maximum m and sum l of each row in registers, the weights
// rounded to the type for the second product and summed as rounded, or (TWO) as two
// parts, rounded weight and rest: in the differential form, whose two sums may all but
// cancel, and for few rows, as the decode holds them (32 single tokens behind
// 2047, 64 heads on 8 of 128 in blocks of 1: 96 us with one part, 105 so; head_dim 256
// for all rows would take the prompts below to 356).  Rows of K and
// V come by 16-byte asynchronous copies from wherever the block table puts
// them, one tile ahead of the products; each row's place is looked up two tiles
// ahead.  Bound by the warps' own latency, four or eight of them on an SM (issue
// 18%, tensor pipe 26%): 4 prompts of 1024 tokens, 16 heads on 4 of 256 320 us, 107
// TFLOP/s; 1 token behind 2047, 32 sequences, 64 heads on 8 of 128 in blocks of 1
// 105 us, 2.6 TB/s.  At head_dim 256 two parts do not fit the registers: a thread stores
// 128 to 134 bytes of its own and loads 592 to 596 (fp16 with one part 40 and 56).
// It is here for head_dim 32 and 256, which chunk_umma.cu is not built for, for scales
// that are not positive and for few rows over blocks that boxes of 8 rows do not fit.
#include "chunk_sched.cuh"

namespace pa {

namespace {

using namespace chunk;

constexpr int kThreads = 128;
constexpr int kKT = 64;                    // cache positions per tile
constexpr int kRows = 64;                  // query rows of all maps

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte offset of 16-byte chunk c of row r in rows of E 16-bit elements,
// permuted so that 8 neighbouring rows' chunks lie in different banks.
template <int E>
__device__ __forceinline__ uint32_t at(int r, int c) {
    constexpr int C = E / 8;               // chunks per row
    const int x = C >= 8 ? r & 7 : C == 4 ? (r >> 1) & 3 : (r >> 2) & 1;
    return (uint32_t)(r * E * 2 + ((c ^ x) << 4));
}

template <typename T>
__device__ __forceinline__ bool non_finite(uint32_t w) {   // of either half
    constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
    return (w & e) == e || ((w >> 16) & e) == e;
}

template <int D, bool DIFF>
struct Layout {
    static constexpr int E = DIFF ? D / 2 : D;
    static constexpr uint32_t kTile = kKT * D * 2;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = kRows * E * 2;             // [2][64][D]
    static constexpr uint32_t kV = kK + 2 * kTile;            // [2][64][D]
    static constexpr uint32_t kStage = kK;                    // end of an item: rows of O in fp32
    static constexpr int kPitch = D + 4;
    static constexpr uint32_t kP = kV + 2 * kTile;            // weights, where V is not finite
    static constexpr uint32_t kSums = kP + kRows * kKT * 4;   // sums of the rows
    static constexpr uint32_t kOff = kSums + kRows * 4;       // [2][64] places of the rows
    static constexpr uint32_t kBad = kOff + 2 * kKT * 8;      // [2] bad table entries of a tile, a bit per row
    static constexpr uint32_t kPre = kBad + 16;
    static constexpr uint32_t kBytes = kPre + (kGroups + 1) * 8;
    static_assert(kRows * kPitch * 4 <= 4 * kTile, "rows of O fit where K and V were");
};

}  // namespace

// TWO: weights go into the second product in two parts, rounded weight and rest.
template <typename T, int D, bool DIFF, bool TWO>
__global__ void __launch_bounds__(kThreads) chunk_mma_kernel(const __grid_constant__ ChunkParams p) {
    using L = Layout<D, DIFF>;
    constexpr int E = L::E, R = DIFF ? kRows / 2 : kRows;
    grid_dependency_wait();
    allow_dependents();
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sb = smem_u32(smem);
    int64_t *off = reinterpret_cast<int64_t *>(smem + L::kOff);
    uint32_t *badm = reinterpret_cast<uint32_t *>(smem + L::kBad);
    float *sums = reinterpret_cast<float *>(smem + L::kSums);
    float *stage = reinterpret_cast<float *>(smem + L::kStage);
    int64_t *pre = reinterpret_cast<int64_t *>(smem + L::kPre);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

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

    const int map = DIFF ? warp >> 1 : 0;
    const int wr = DIFF ? (warp & 1) * 16 : warp * 16;         // the warp's first row in its map
    do {
        const Item x = it.x;
        const int n0 = x.i * R, nrows = min(R, x.cnt * p.G - n0);
        const int tmin = (int)by_group(p, n0), tmax = (int)by_group(p, n0 + nrows - 1);
        const int need_lo = p.window > 0 ? max(0, x.pos + tmin - p.window + 1) : 0, need_hi = x.pos + tmax;
        const int wlo_max = p.window > 0 ? max(0, x.pos + tmax - p.window + 1) : 0;
        // query rows: row m * R + r holds map m of row r
        for (int c = tid; c < kRows * (E / 8); c += kThreads) {
            const int row = c / (E / 8), ch = c % (E / 8), r = row % R, m = row / R, n = n0 + r;
            const T *src = reinterpret_cast<const T *>(p.q);
            if (r < nrows)
                src += ((int64_t)x.b * p.T + by_group(p, n)) * p.q_stride +
                       (int64_t)(x.hk * p.G + (n - (int)by_group(p, n) * p.G)) * D + m * E + ch * 8;
            cp16(sb + L::kQ + at<E>(row, ch), src, r < nrows);
        }
        // places of the rows of tile k: -1 not needed, -2 bad
        auto look_up = [&](int k) -> int64_t {
            const int t = (x.lo + k) * kKT + tid;
            if (tid >= kKT || k >= x.k1 || t < need_lo || t > need_hi) return -1;
            const int64_t o = row_offset(p, x.b, x.hk, t, D * 2);
            return o < 0 ? -2 : o;
        };
        auto put_places = [&](int k, int64_t o) {
            if (tid < kKT) {
                off[(k & 1) * kKT + tid] = o;
                const uint32_t bad = __ballot_sync(0xffffffffu, o == -2);
                if (lane == 0) badm[(k & 1) * 2 + warp] = bad;
            }
        };
        auto copy_tile = [&](int k) {
            if (k < x.k1) {
                const uint32_t kd = sb + L::kK + (k & 1) * L::kTile, vd = sb + L::kV + (k & 1) * L::kTile;
                for (int c = tid; c < kKT * (D / 8); c += kThreads) {
                    const int row = c / (D / 8), ch = c % (D / 8);
                    const int64_t o = off[(k & 1) * kKT + row];
                    const int64_t byte = (o < 0 ? 0 : o) + ch * 16;
                    cp16(kd + at<D>(row, ch), p.k_pool + byte, o >= 0);
                    cp16(vd + at<D>(row, ch), p.v_pool + byte, o >= 0);
                }
            }
            cp_commit();
        };
        put_places(x.k0, look_up(x.k0));
        __syncthreads();
        copy_tile(x.k0);
        int64_t ahead = look_up(x.k0 + 1);

        // this thread's two rows of its map
        int row_lo[2], row_hi[2];
        bool row_bad[2] = {false, false};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = wr + lane / 4 + 8 * h;
            const int pos = x.pos + (int)by_group(p, n0 + r);
            row_hi[h] = r < nrows ? pos : INT32_MAX;           // rows that are not there may see anything
            row_lo[h] = r < nrows && p.window > 0 ? max(0, pos - p.window + 1) : 0;
        }
        float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

        for (int k = x.k0; k < x.k1; ++k) {
            put_places(k + 1, ahead);
            __syncthreads();
            copy_tile(k + 1);
            ahead = look_up(k + 2);
            cp_wait<1>();
            __syncthreads();
            const uint32_t kb = sb + L::kK + (k & 1) * L::kTile, vb = sb + L::kV + (k & 1) * L::kTile;
            const int t0 = (x.lo + k) * kKT;
            float s[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll
            for (int kk = 0; kk < E / 16; ++kk) {
                uint32_t a[4];
                ldsm_x4(sb + L::kQ + at<E>(warp * 16 + (lane & 15), kk * 2 + (lane >> 4)), a[0], a[1], a[2], a[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4(kb + at<D>(j * 16 + (lane & 7) + ((lane >> 4) << 3), map * (E / 8) + kk * 2 + ((lane >> 3) & 1)),
                            b0, b1, b2, b3);
                    MmaOp<T>::run(s[2 * j], a, b0, b1);
                    MmaOp<T>::run(s[2 * j + 1], a, b2, b3);
                }
            }
            // weights
            const bool partial = t0 < wlo_max || t0 + kKT - 1 > x.pos + tmin;
            const uint64_t bad = (uint64_t)badm[(k & 1) * 2 + 1] << 32 | badm[(k & 1) * 2];
            float alpha[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float mx = m[h];
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int t = t0 + i * 8 + (lane & 3) * 2 + j;
                        float v = s[i][2 * h + j] * p.scale_log2;
                        if (partial && (t < row_lo[h] || t > row_hi[h])) v = -INFINITY;
                        s[i][2 * h + j] = v;
                        mx = fmaxf(mx, v);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float ref = mx == -INFINITY ? 0.f : mx;
                alpha[h] = ex2_approx(m[h] - ref);
                m[h] = mx;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float &w0 = s[i][2 * h], &w1 = s[i][2 * h + 1];
                    w0 = ex2_approx(w0 - ref);
                    w1 = ex2_approx(w1 - ref);
                    // one part: exactly the weights that the product uses, in the sum too
                    if (!TWO) Elem<T>::unpack2(Elem<T>::pack2(w0, w1), w0, w1);
                    sum += w0;
                    sum += w1;
                }
                l[h] = l[h] * alpha[h] + sum;
                if (bad != 0) {
                    const int a = max(0, row_lo[h] - t0), e = min(kKT - 1, row_hi[h] - t0);
                    if (a <= e && ((bad >> a) << a << (kKT - 1 - e)) != 0) row_bad[h] = true;
                }
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] *= alpha[j >> 1];
            // where rows of a tile see different positions, a value that is not
            // finite must not reach the rows that do not see it, as 0 times it would
            bool odd = false;
            if (partial) {
                for (int c = tid; c < (int)(L::kTile / 16); c += kThreads) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(smem + L::kV + (k & 1) * L::kTile + c * 16);
                    odd |= non_finite<T>(v.x) || non_finite<T>(v.y) || non_finite<T>(v.z) || non_finite<T>(v.w);
                }
                odd = __syncthreads_or(odd);
            }
            if (!odd) {
#pragma unroll
                for (int kk = 0; kk < kKT / 16; ++kk) {
                    uint32_t a[4], rest[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const float (&w)[4] = s[2 * kk + (h >> 1)];
                        const float w0 = w[2 * (h & 1)], w1 = w[2 * (h & 1) + 1];
                        a[h] = Elem<T>::pack2(w0, w1);
                        if constexpr (TWO) {
                            float r0, r1;
                            Elem<T>::unpack2(a[h], r0, r1);
                            rest[h] = Elem<T>::pack2(w0 - r0, w1 - r1);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4_trans(vb + at<D>(kk * 16 + (lane & 15), j * 2 + (lane >> 4)), b0, b1, b2, b3);
                        MmaOp<T>::run(o[2 * j], a, b0, b1);
                        MmaOp<T>::run(o[2 * j + 1], a, b2, b3);
                        if constexpr (TWO) {
                            MmaOp<T>::run(o[2 * j], rest, b0, b1);
                            MmaOp<T>::run(o[2 * j + 1], rest, b2, b3);
                        }
                    }
                }
            } else {
                float *pw = reinterpret_cast<float *>(smem + L::kP) + warp * 16 * kKT;
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<float2 *>(pw + (lane / 4 + 8 * h) * kKT + i * 8 + (lane & 3) * 2) =
                            make_float2(s[i][2 * h], s[i][2 * h + 1]);
                __syncwarp();
#pragma unroll 1
                for (int t = 0; t < kKT; ++t) {
                    float w[2];
                    bool sees[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        w[h] = pw[(lane / 4 + 8 * h) * kKT + t];
                        sees[h] = t0 + t >= row_lo[h] && t0 + t <= row_hi[h];
                    }
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const uint32_t v = *reinterpret_cast<const uint32_t *>(smem + (vb - sb) + at<D>(t, i) + (lane & 3) * 4);
                        float v0, v1;
                        Elem<T>::unpack2(v, v0, v1);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (sees[h]) {
                                o[i][2 * h] += w[h] * v0;
                                o[i][2 * h + 1] += w[h] * v1;
                            }
                    }
                }
                __syncwarp();
            }
            __syncthreads();
        }
        cp_wait<0>();

        bool any_bad = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (row_bad[h]) l[h] = -1.f;
            any_bad |= row_bad[h] && wr + lane / 4 + 8 * h < nrows;
        }
        if (any_bad && (lane & 3) == 0) report(p.err_word, PA_DEVERR_BAD_BLOCK);
        const bool cut = it.cut();
        float *rec = p.records + ((int64_t)blockIdx.x * 2 + (x.k0 == 0)) * p.rec_floats;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = warp * 16 + lane / 4 + 8 * h;
            const float inv = cut ? 1.f : l[h] == 0.f ? 0.f : 1.f / l[h];
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const int c = i * 8 + (lane & 3) * 2;
                float *dst = cut ? record_at(rec, kRows, row, c) : stage + row * L::kPitch + c;
                *reinterpret_cast<float2 *>(dst) = make_float2(o[i][2 * h] * inv, o[i][2 * h + 1] * inv);
            }
            if ((lane & 3) == 0) {
                if (cut) {
                    rec[kRows * D + row] = m[h];
                    rec[kRows * D + kRows + row] = l[h];
                } else {
                    sums[row] = l[h];
                }
            }
        }
        __syncthreads();
        if (!cut) {
            for (int r = warp; r < nrows; r += kThreads / 32) {
                const int n = n0 + r;
                finish_row<T, D, DIFF>(p, stage + r * L::kPitch + lane * (D / 32),
                                       stage + (kRows / 2 + r) * L::kPitch + lane * (D / 32),
                                       sums[r] < 0.f || (DIFF && sums[kRows / 2 + r] < 0.f), (int64_t)x.b * p.T + by_group(p, n),
                                       x.hk * p.G + n - (int)by_group(p, n) * p.G);
            }
            __syncthreads();
        }
    } while (it.next(p));
}

namespace {

template <typename T, int D, bool DIFF, bool TWO>
cudaError_t plan_one(ChunkPlan *plan) {
    static std::atomic<int> limit[64];
    static std::atomic<int64_t> cache[64];
    auto kern = chunk_mma_kernel<T, D, DIFF, TWO>;
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
    plan->two_parts = TWO;
    plan->rec_floats = chunk_rec_floats(kRows, D);
    return cudaSuccess;
}

template <typename T, int D, bool DIFF, bool TWO>
cudaError_t launch_one(const ChunkParams &p, const ChunkPlan &plan, cudaStream_t stream) {
    return launch_clustered(chunk_mma_kernel<T, D, DIFF, TWO>, plan.grid, kThreads, Layout<D, DIFF>::kBytes, 1, stream, p);
}

template <typename T, bool DIFF, bool TWO, typename F>
cudaError_t with_dim(int head_dim, F f) {
    switch (head_dim) {
        case 32: return f.template operator()<T, 32, DIFF, TWO>();
        case 64: return f.template operator()<T, 64, DIFF, TWO>();
        case 128: return f.template operator()<T, 128, DIFF, TWO>();
        case 256: return f.template operator()<T, 256, DIFF, TWO>();
    }
    return cudaErrorInvalidValue;
}
template <typename T, typename F>
cudaError_t with_form(int head_dim, bool diff, bool two, F f) {
    if (diff) return with_dim<T, true, true>(head_dim, f);
    return two ? with_dim<T, false, true>(head_dim, f) : with_dim<T, false, false>(head_dim, f);
}
template <typename F>
cudaError_t with_kernel(int dtype, int head_dim, bool diff, bool two, F f) {
    if (dtype == PA_F16) return with_form<__half>(head_dim, diff, two, f);
    if (dtype == PA_BF16) return with_form<__nv_bfloat16>(head_dim, diff, two, f);
    return cudaErrorInvalidValue;
}

struct Planner {
    ChunkPlan *plan;
    template <typename T, int D, bool DIFF, bool TWO>
    cudaError_t operator()() const { return plan_one<T, D, DIFF, TWO>(plan); }
};
struct Launcher {
    const ChunkParams &p;
    const ChunkPlan &plan;
    cudaStream_t stream;
    template <typename T, int D, bool DIFF, bool TWO>
    cudaError_t operator()() const { return launch_one<T, D, DIFF, TWO>(p, plan, stream); }
};

}  // namespace

cudaError_t plan_chunk_mma(int dtype, int head_dim, bool diff, bool two_parts, ChunkPlan *plan) {
    return with_kernel(dtype, head_dim, diff, two_parts, Planner{plan});
}
cudaError_t launch_chunk_mma(int dtype, int head_dim, const ChunkParams &p, const ChunkPlan &plan, cudaStream_t stream) {
    return with_kernel(dtype, head_dim, plan.maps == 2, plan.two_parts, Launcher{p, plan, stream});
}

}  // namespace pa
