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
// for prompts (8 of 900 to 2047 tokens, 64 + 8 heads of 128, bf16: 554 MB in 89 us,
// 6.2 TB/s, 92% of the copy rate) and by launch and the dependent loads (position,
// table entry and cosines) for single tokens (1: 1.9 us; 256 of 32 + 32 heads: 2.9
// us).  Into the 4-bit cache keys and values take three times their bytes' time: the
// arithmetic of the codes (f16 prompts, 32 + 8 heads: 28.3 us, 13 of them theirs).
//
// D/8 lanes hold a row, 8 elements each in two chunks of 4.  With pairs (i, i + R/2)
// a lane takes chunk i and chunk i + R/2 (kSplit): each chunk of a row is still read
// in whole 128-byte lines, both elements of a pair are in one lane, and its 4
// cosines and sines serve both chunks.  With pairs (2i, 2i + 1), or none, the chunks
// are neighbours.  Only where the halves of R cut a 4-bit group of 16 (R not a
// multiple of 32) are neighbouring chunks kept and the other elements of the pairs
// fetched by shuffles (kShuffle).
//
// A warp takes a run of the queries of one token, or of its keys with the values
// beside them: up to 8 rows a lane, all of whose loads are issued at once, before
// the positions, table entries and cosines that they do not depend on.
// Products (two at a time, f32x2) and sums are rounded separately: the results are
// those of the stated formula operation by operation, and so are the 4-bit codes.
//
// Quotients of the 4-bit scheme: q = x r, then q - r (q t - x), with r the
// correctly rounded reciprocal of t, is the correctly rounded quotient (P. W.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) where nothing over- or underflows; a group with a NaN or a
// magnitude that could overflow takes IEEE divisions instead.
#include "fp4.cuh"
#include "pa_rope_fp4.h"

namespace pa {

// Warps per CTA: small ones, whose slots are free again as soon as both are done
// (8 prompts of 900 to 2047 tokens, 64 + 8 heads of 128, bf16: 97.8 us at 8, 91.5 at
// 4, 89.3 at 2, 90.5 at 1, with as many registers).
constexpr int kRopeWarps = 2;
constexpr int kRopeThreads = kRopeWarps * 32;
enum RopeMode { kSplit, kNeighbours, kShuffle };

// --- two fp32 values in one register pair -------------------------------------
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// Sums one by one: a packed sum of packed products comes out fused, whatever their
// rounding modifiers and the compiler's flags say (a quarter of the rotated fp32
// values differed in the last bit; 88.4 us so, 89.7 with scalar sums, 93.2 with
// scalar products too, on 8 bf16 prompts).
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// 4 elements of T: as they are in memory, and as fp32 pairs.
template <typename T>
struct Chunk {
    uint2 v;
    __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void zero() { v = make_uint2(0, 0); }
    __device__ __forceinline__ void unpack(float2 (&x)[2]) const {
        Elem<T>::unpack2(v.x, x[0].x, x[0].y);
        Elem<T>::unpack2(v.y, x[1].x, x[1].y);
    }
    __device__ __forceinline__ void pack(const float2 (&x)[2]) {
        v = make_uint2(Elem<T>::pack2(x[0].x, x[0].y), Elem<T>::pack2(x[1].x, x[1].y));
    }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<uint2 *>(p) = v; }
    static __device__ __forceinline__ void load2(const T *p, Chunk &a, Chunk &b) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        a.v = make_uint2(w.x, w.y);
        b.v = make_uint2(w.z, w.w);
    }
    static __device__ __forceinline__ void store2(T *p, const Chunk &a, const Chunk &b) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(a.v.x, a.v.y, b.v.x, b.v.y);
    }
};
template <>
struct Chunk<float> {
    float4 v;
    __device__ __forceinline__ void load(const float *p) { v = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void unpack(float2 (&x)[2]) const { x[0] = make_float2(v.x, v.y), x[1] = make_float2(v.z, v.w); }
    __device__ __forceinline__ void pack(const float2 (&x)[2]) { v = make_float4(x[0].x, x[0].y, x[1].x, x[1].y); }
    __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = v; }
    static __device__ __forceinline__ void load2(const float *p, Chunk &a, Chunk &b) { a.load(p), b.load(p + 4); }
    static __device__ __forceinline__ void store2(float *p, const Chunk &a, const Chunk &b) { a.store(p), b.store(p + 4); }
};

// --- 4-bit groups ---------------------------------------------------------------
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if one is
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float largest(const float2 (&x)[2]) {
    return max_nan(max_nan(fabsf(x[0].x), fabsf(x[0].y)), max_nan(fabsf(x[1].x), fabsf(x[1].y)));
}
// The factor of one half of the cache: 6 g, its reciprocal, and the magnitude
// up to which no quotient overflows.
struct Factor {
    float g, six_g, r6, limit;
};
__device__ __forceinline__ Factor factor_of(float g) {
    Factor f;
    f.g = g;
    f.six_g = __fmul_rn(6.f, g);
    f.r6 = __frcp_rn(f.six_g);
    f.limit = f.six_g * 1024.f;
    return f;
}
// The E4M3 code of a group with largest magnitude a, and the value t that its
// codes are multiples of; a within the factor's limit (Markstein), or any.
__device__ __forceinline__ float group_value(uint32_t code, const Factor &f) {
    return __fmul_rn(f16x2_to_float2(e4m3x2_to_f16x2(code)).x, f.g);
}
__device__ __forceinline__ uint32_t group_scale(float a, const Factor &f) {
    const float q = __fmul_rn(a, f.r6);
    return f32_to_e4m3(__fmaf_rn(__fmaf_rn(-q, f.six_g, a), f.r6, q));
}
__device__ __forceinline__ uint32_t group_scale_any(float a, const Factor &f) { return f32_to_e4m3(__fdiv_rn(a, f.six_g)); }
// Two bytes of codes of x / t, r the reciprocal of t > 0; or any x and t.
__device__ __forceinline__ uint32_t pack_codes(const float2 (&y)[2]) {
    return f32x2_to_e2m1x2(y[0].x, y[0].y) | f32x2_to_e2m1x2(y[1].x, y[1].y) << 8;
}
__device__ __forceinline__ uint32_t group_codes(const float2 (&x)[2], float t, float r) {
    float2 y[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {                  // (q t - x) (-r) + q keeps the sign of a zero
        const float2 minus_x = mul2(x[j], both(-1.f));
        y[j] = mul2(minus_x, both(-r));
        y[j] = fma2(fma2(y[j], both(t), minus_x), both(-r), y[j]);
    }
    return pack_codes(y);
}
__device__ __forceinline__ uint32_t group_codes_any(const float2 (&x)[2], float t) {
    float2 y[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        y[j].x = x[j].x == x[j].x ? __fdiv_rn(x[j].x, t) : 0.f;
        y[j].y = x[j].y == x[j].y ? __fdiv_rn(x[j].y, t) : 0.f;
    }
    return t > 0.f ? pack_codes(y) : 0;
}

// Quantise a row: chunks x and y of this lane.  A group of 16 is 4 lanes' chunks x
// or chunks y if they are `apart` (SPLIT only), else 2 lanes' both chunks.  The
// scale of a lane pair's two groups is found by one lane of the pair each.  Codes
// go to cd + da / 2, cd + db / 2, scales to sd, if `mine`.
template <bool SPLIT>
__device__ __forceinline__ void store_fp4(const float2 (&x)[2], const float2 (&y)[2], const Factor &f, bool apart, bool mine,
                                          int sub, int da, int db, uint8_t *cd, uint8_t *sd) {
    const unsigned all = 0xffffffffu;
    float mx = largest(x), my = largest(y);
    if (!apart) mx = my = max_nan(mx, my);
    mx = max_nan(mx, __shfl_xor_sync(all, mx, 1));
    if constexpr (SPLIT) {
        my = max_nan(my, __shfl_xor_sync(all, my, 1));
        const float fx = __shfl_xor_sync(all, mx, 2), fy = __shfl_xor_sync(all, my, 2);
        if (apart) mx = max_nan(mx, fx), my = max_nan(my, fy);
    }
    const bool odd = (sub & 1) != 0;
    uint32_t code, wx, wy;                         // of this lane's group; the codes of both chunks
    if (__all_sync(all, mx <= f.limit && (!SPLIT || my <= f.limit))) {
        code = group_scale(SPLIT && odd ? my : mx, f);
        const float t = group_value(code, f), r = t > 0.f ? __frcp_rn(t) : 0.f;
        float tx = t, ty = t, rx = r, ry = r;
        if constexpr (SPLIT) {
            const float ot = __shfl_xor_sync(all, t, 1), orr = __shfl_xor_sync(all, r, 1);
            tx = odd ? ot : t, ty = odd ? t : ot;
            rx = odd ? orr : r, ry = odd ? r : orr;
        }
        wx = tx > 0.f ? group_codes(x, tx, rx) : 0;
        wy = ty > 0.f ? group_codes(y, ty, ry) : 0;
    } else {                                       // a NaN counts as 0
        float vx = fmaxf(fmaxf(fabsf(x[0].x), fabsf(x[0].y)), fmaxf(fmaxf(fabsf(x[1].x), fabsf(x[1].y)), 0.f));
        float vy = fmaxf(fmaxf(fabsf(y[0].x), fabsf(y[0].y)), fmaxf(fmaxf(fabsf(y[1].x), fabsf(y[1].y)), 0.f));
        if (!apart) vx = vy = fmaxf(vx, vy);
        vx = fmaxf(vx, __shfl_xor_sync(all, vx, 1));
        vy = fmaxf(vy, __shfl_xor_sync(all, vy, 1));
        const float fx = __shfl_xor_sync(all, vx, 2), fy = __shfl_xor_sync(all, vy, 2);
        if (apart) vx = fmaxf(vx, fx), vy = fmaxf(vy, fy);
        const uint32_t cx = group_scale_any(vx, f), cy = group_scale_any(vy, f);
        wx = group_codes_any(x, group_value(cx, f));
        wy = group_codes_any(y, group_value(cy, f));
        code = SPLIT && odd ? cy : cx;
    }
    if (!mine) return;
    if (apart) {
        *reinterpret_cast<uint16_t *>(cd + da / 2) = (uint16_t)wx;
        *reinterpret_cast<uint16_t *>(cd + db / 2) = (uint16_t)wy;
        if (sub % 4 < 2) sd[(odd ? db : da) / 16] = (uint8_t)code;
    } else {
        *reinterpret_cast<uint32_t *>(cd + da / 2) = wx | wy << 16;
        if (!odd) sd[da / 16] = (uint8_t)code;
    }
}

// grid: x = kRopeWarps tokens of the padded batch each, y = run: of kv_run
// iterations of keys and values, then of q_run iterations of queries (at most
// KB and QB), so that the warps of a CTA do the same (runs of a token side by
// side instead: equal).
// Iterations of queries a run has at most, as many as keep their registers; half
// as many of keys, with their values (half of these: 100.1 us for 89.3 on the bf16
// prompts, 32.5 for 28.3 on f16 ones into the 4-bit cache, 104.4 for 98.5 on fp32 ones
// of 32 + 8 heads and 63.2 for 47.9 on such into the 4-bit cache; fp32 as 16-bit types:
// 99.7 and 51.6).
template <typename T>
constexpr int kRopeBatch = sizeof(T) == 2 ? 8 : 4;
// CTAs per SM that registers have to do for (the bf16 prompts above: 93.1 us at 12,
// 89.3 at 13 and 14, 97.5 at 15; f16 ones into the 4-bit cache: 28.9 at 10, 28.3 at 11,
// 28.1 at 12, 29.0 at 13; fp32: 98.5 from 8 to 12, into the 4-bit cache 53.5 at 8, 47.9
// at 10, 45.9 at 12).  The 16-bit kernels of the 4-bit cache, which would take up to 96
// registers, spill at 80: a thread stores 16 to 24 bytes and loads 52 to 60, with pairs
// by shuffles 52 to 56 and 216 to 220; so do those of head_dim 256 with pairs in
// halves, 4 and 8 bytes at 72.
template <typename T, bool FP4>
constexpr int kRopeCtas = sizeof(T) == 4 ? 10 : FP4 ? 11 : 14;

template <typename T, int D, bool FP4, RopeMode MODE>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas<T, FP4>)
rope_append_kernel(const __grid_constant__ RopeAppendParams p, const int q_run, const int kv_run, const int kv_runs) {
    grid_dependency_wait();
    allow_dependents();
    constexpr int LPR = D / 8;                     // lanes per row
    constexpr int RPW = 32 / LPR;                  // rows per iteration of a warp
    constexpr int QB = kRopeBatch<T>, KB = QB / 2;
    const int64_t token = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    if (token >= (int64_t)p.B * p.T) return;
    const int b = p.T == 1 ? (int)token : (int)((uint32_t)token / (uint32_t)p.T);
    const int t = (int)(token - (int64_t)b * p.T);
    const int n = p.counts != nullptr ? __ldg(p.counts + b) : p.T;
    const int32_t start = __ldg(p.positions + b);

    const int lane = threadIdx.x & 31, sub = lane % LPR, lr = lane / LPR;
    const int HQ = p.q != nullptr ? p.H : 0;
    const int nq = (HQ + RPW - 1) / RPW, nk = (p.Hkv + RPW - 1) / RPW;   // iterations over queries, over keys
    const bool queries = (int)blockIdx.y >= kv_runs;
    const int from = queries ? ((int)blockIdx.y - kv_runs) * q_run : (int)blockIdx.y * kv_run;
    const int count = queries ? min(q_run, nq - from) : min(kv_run, nk - from);
    const int heads = queries ? HQ : p.Hkv;
    // this lane's chunks, and whether they are rotated
    const bool reporter = t == 0 && blockIdx.y == 0 && lane == 0;
    const bool turn = sub < p.R / 8;
    const bool apart = MODE == kSplit && turn;
    const int da = apart ? 4 * sub : 8 * sub, db = apart ? p.R / 2 + 4 * sub : 8 * sub + 4;
    const int half = p.R / 16;                     // kShuffle: lanes between the two elements of a pair
    const int partner = MODE == kShuffle && turn ? lane + (sub < half ? half : -half) : lane;

    // padding is not read; a first token's row is memory whatever the count
    if (t > 0 && n >= 0 && n <= p.T && t >= n) return;
    // the rows: queries in the first QB places, or KB of keys and KB of values
    Chunk<T> ra[QB], rb[QB];
    {
        const T *src = (queries ? reinterpret_cast<const T *>(p.q) + token * p.q_stride
                                : reinterpret_cast<const T *>(p.k) + token * p.k_stride) + (int64_t)(from * RPW + lr) * D;
        const T *src_v = reinterpret_cast<const T *>(p.v) + token * p.v_stride + (int64_t)(from * RPW + lr) * D;
#pragma unroll
        for (int u = 0; u < QB; ++u) {
            const int i = queries || u < KB ? u : u - KB;
            const T *row = (queries || u < KB ? src : src_v) + i * RPW * D;
            ra[u].zero();
            rb[u].zero();
            if (i < count && (queries || u < 2 * KB) && (from + i) * RPW + lr < heads) {
                // values that are quantised: neighbouring chunks, one group a lane
                if (MODE == kSplit && !(FP4 && !queries && u >= KB)) ra[u].load(row + da), rb[u].load(row + db);
                else Chunk<T>::load2(row + 8 * sub, ra[u], rb[u]);
            }
        }
    }
    if (n < 0 || n > p.T) {
        if (reporter) report(p.err_word, PA_DEVERR_BAD_LEN);
        return;
    }
    const bool bad_pos = start < 0 || (int64_t)start + n > (int64_t)p.MB * p.bs ||
                         (p.R > 0 && (int64_t)start + n > (int64_t)p.max_position);
    if (bad_pos && reporter) report(p.err_word, PA_DEVERR_BAD_POS);
    if (t >= n) return;
    if (bad_pos) {                             // zeros for the queries, nothing for the cache
        Chunk<T> z;
        z.zero();
        for (int i = 0; i < (queries ? count : 0); ++i) {
            const int h = (from + i) * RPW + lr;
            if (h < HQ) Chunk<T>::store2(reinterpret_cast<T *>(p.q_out) + (token * p.H + h) * D + 8 * sub, z, z);
        }
        return;
    }
    const int32_t pos = start + t;
    const int32_t bj = p.bs_shift >= 0 ? pos >> p.bs_shift : pos / p.bs, slot = pos - bj * p.bs;
    const int64_t blk = queries ? 0 : __ldg(p.block_table + (int64_t)b * p.MB + bj);
    // cosines and sines: of pairs of elements, -sine first where the formula subtracts
    float2 c[MODE == kSplit ? 2 : 4], s[MODE == kSplit ? 2 : 4], ns[2];
    if (turn) {
        const float *cs = p.cos_sin + (int64_t)pos * p.R;
        if constexpr (MODE == kShuffle) {
            const int i = sub < half ? 8 * sub : 8 * sub - p.R / 2;
            float c8[8], s8[8];
            load8(cs + i, c8);
            load8(cs + p.R / 2 + i, s8);
            const float sign = sub < half ? -1.f : 1.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c[j] = make_float2(c8[2 * j], c8[2 * j + 1]);
                s[j] = make_float2(sign * s8[2 * j], sign * s8[2 * j + 1]);
            }
        } else {
            const float4 c4 = *reinterpret_cast<const float4 *>(cs + 4 * sub);
            const float4 s4 = *reinterpret_cast<const float4 *>(cs + p.R / 2 + 4 * sub);
            if constexpr (MODE == kSplit) {
                c[0] = make_float2(c4.x, c4.y), c[1] = make_float2(c4.z, c4.w);
                s[0] = make_float2(s4.x, s4.y), s[1] = make_float2(s4.z, s4.w);
                ns[0] = make_float2(-s4.x, -s4.y), ns[1] = make_float2(-s4.z, -s4.w);
            } else {
                c[0] = both(c4.x), c[1] = both(c4.y), c[2] = both(c4.z), c[3] = both(c4.w);
                s[0] = make_float2(-s4.x, s4.x), s[1] = make_float2(-s4.y, s4.y);
                s[2] = make_float2(-s4.z, s4.z), s[3] = make_float2(-s4.w, s4.w);
            }
        }
    }
    const void *weight = queries ? p.q_weight : p.k_weight;
    float2 wa[2], wb[2];
    if (weight != nullptr) {
        Chunk<T> w0, w1;
        w0.load(reinterpret_cast<const T *>(weight) + da);
        w1.load(reinterpret_cast<const T *>(weight) + db);
        w0.unpack(wa);
        w1.unpack(wb);
    }
    // norm and rotation of a row
    auto turned = [&](float2 (&x)[2], float2 (&y)[2]) {
        if (weight != nullptr) {
            float2 q2 = mul2(x[0], x[0]);
            q2 = fma2(x[1], x[1], q2);
            q2 = fma2(y[0], y[0], q2);
            q2 = fma2(y[1], y[1], q2);
            float sq = q2.x + q2.y;
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
            const float2 rstd = both(__frsqrt_rn(__fadd_rn(sq * (1.f / D), p.eps)));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                x[j] = mul2(mul2(x[j], rstd), wa[j]);
                y[j] = mul2(mul2(y[j], rstd), wb[j]);
            }
        }
        if constexpr (MODE == kShuffle) {
            float2 ox[2], oy[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                ox[j].x = __shfl_sync(0xffffffffu, x[j].x, partner);
                ox[j].y = __shfl_sync(0xffffffffu, x[j].y, partner);
                oy[j].x = __shfl_sync(0xffffffffu, y[j].x, partner);
                oy[j].y = __shfl_sync(0xffffffffu, y[j].y, partner);
            }
            if (turn) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    x[j] = add2(mul2(x[j], c[j]), mul2(ox[j], s[j]));
                    y[j] = add2(mul2(y[j], c[j + 2]), mul2(oy[j], s[j + 2]));
                }
            }
        } else if (turn) {
            if constexpr (MODE == kSplit) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 v = x[j], w = y[j];
                    x[j] = add2(mul2(v, c[j]), mul2(w, ns[j]));
                    y[j] = add2(mul2(w, c[j]), mul2(v, s[j]));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    x[j] = add2(mul2(x[j], c[j]), mul2(make_float2(x[j].y, x[j].x), s[j]));
                    y[j] = add2(mul2(y[j], c[j + 2]), mul2(make_float2(y[j].y, y[j].x), s[j + 2]));
                }
            }
        }
    };
    auto put = [&](T *dst, const Chunk<T> &ca, const Chunk<T> &cb) {
        if constexpr (MODE == kSplit) ca.store(dst + da), cb.store(dst + db);
        else Chunk<T>::store2(dst + da, ca, cb);
    };
    if (queries) {
        T *dst = reinterpret_cast<T *>(p.q_out) + (token * p.H + from * RPW + lr) * D;
#pragma unroll
        for (int u = 0; u < QB; ++u) {
            if (u >= count) break;             // the same for the whole warp
            float2 x[2], y[2];
            ra[u].unpack(x);
            rb[u].unpack(y);
            turned(x, y);
            if ((from + u) * RPW + lr < HQ) {
                ra[u].pack(x);
                rb[u].pack(y);
                put(dst + u * RPW * D, ra[u], rb[u]);
            }
        }
        return;
    }

    const bool to_cache = blk >= 0 && blk < p.num_blocks;
    if (!to_cache && blockIdx.y == 0 && lane == 0) report(p.err_word, PA_DEVERR_BAD_BLOCK);
    const int64_t first = (int64_t)(from * RPW + lr) * p.bs + slot;   // this lane's first row in the block
    if constexpr (FP4) {
        const Factor fk = factor_of(p.k_g), fv = factor_of(p.v_g);
        const int64_t code_step = (int64_t)RPW * p.bs * (D / 2), scale_step = (int64_t)RPW * p.bs * (D / 16);
        uint8_t *cd = reinterpret_cast<uint8_t *>(p.k_pool) + blk * p.block_stride_bytes + first * (D / 2);
        uint8_t *sd = p.scales + (blk * 2 * p.Hkv * p.bs + first) * (D / 16);
        // one copy of the code for the keys, one for the values: the rows move up to it
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
            float2 x[2], y[2];
            ra[0].unpack(x);
            rb[0].unpack(y);
            turned(x, y);
            store_fp4<MODE == kSplit>(x, y, fk, apart, to_cache && (from + i) * RPW + lr < p.Hkv, sub, da, db, cd + i * code_step,
                                      sd + i * scale_step);
#pragma unroll
            for (int j = 0; j + 1 < KB; ++j) ra[j] = ra[j + 1], rb[j] = rb[j + 1];
        }
        cd = reinterpret_cast<uint8_t *>(p.v_pool) + blk * p.block_stride_bytes + first * (D / 2);
        sd += (int64_t)p.Hkv * p.bs * (D / 16);
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
            float2 x[2], y[2];
            ra[KB].unpack(x);
            rb[KB].unpack(y);
            store_fp4<false>(x, y, fv, false, to_cache && (from + i) * RPW + lr < p.Hkv, sub, 8 * sub, 8 * sub + 4,
                             cd + i * code_step, sd + i * scale_step);
#pragma unroll
            for (int j = KB; j + 1 < 2 * KB; ++j) ra[j] = ra[j + 1], rb[j] = rb[j + 1];
        }
    } else {
#pragma unroll
        for (int u = 0; u < 2 * KB; ++u) {
            const int i = u < KB ? u : u - KB;
            if (i >= count) continue;              // the same for the whole warp
            if (u < KB) {                          // values go as they came, to the last bit
                float2 x[2], y[2];
                ra[u].unpack(x);
                rb[u].unpack(y);
                turned(x, y);
                ra[u].pack(x);
                rb[u].pack(y);
            }
            if (to_cache && (from + i) * RPW + lr < p.Hkv)
                put(reinterpret_cast<T *>((u < KB ? p.k_pool : p.v_pool) + blk * p.block_stride_bytes) +
                        (first + (int64_t)i * RPW * p.bs) * D,
                    ra[u], rb[u]);
        }
    }
}

template <typename T, int D, bool FP4, RopeMode MODE>
static cudaError_t launch_mode(const RopeAppendParams &p, cudaStream_t stream) {
    constexpr int RPW = 32 / (D / 8), QB = kRopeBatch<T>, KB = QB / 2;
    const int nq = ((p.q != nullptr ? p.H : 0) + RPW - 1) / RPW, nk = (p.Hkv + RPW - 1) / RPW;
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    // Rows per run: as many as are loaded at once, which amortises what a token
    // costs; fewer for few tokens, the longer of the two runs first (a quantised
    // row takes about as long as four others), until every SM has 12 warps at most
    // (1 token: 3.2 us with full runs, 1.9 so; 64 tokens into the 4-bit cache: 5.0 and
    // 2.9, 3.3 where SMs may have 16 or 24; 256 tokens: 2.8, 3.2 at 24).
    const int64_t tokens = (int64_t)p.B * p.T, most = (int64_t)sms * 12;
    int q_run = QB, kv_run = KB;
    auto fits = [&](int q, int kv) { return q >= 1 && kv >= 1 && tokens * ((nq + q - 1) / q + (nk + kv - 1) / kv) <= most; };
    for (;;) {
        const bool kv_first = kv_run * (FP4 ? 4 : 2) >= q_run, kv = fits(q_run, kv_run / 2), q = fits(q_run / 2, kv_run);
        if (kv && (kv_first || !q)) kv_run /= 2;
        else if (q) q_run /= 2;
        else break;
    }
    const int kv_runs = (nk + kv_run - 1) / kv_run, runs = (nq + q_run - 1) / q_run + kv_runs;
    if (runs > 65535) return cudaErrorInvalidValue;
    const int64_t gx = (tokens + kRopeWarps - 1) / kRopeWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)gx, (unsigned)runs, 1);
    cfg.blockDim = dim3(kRopeThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = PA_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_append_kernel<T, D, FP4, MODE>, p, q_run, kv_run, kv_runs);
}

template <typename T, int D, bool FP4>
static cudaError_t launch_one(const RopeAppendParams &p, cudaStream_t stream) {
    if (p.R == 0 || p.pairs) return launch_mode<T, D, FP4, kNeighbours>(p, stream);
    if constexpr (FP4) {
        if (p.R % 32 != 0) return launch_mode<T, D, FP4, kShuffle>(p, stream);
    }
    return launch_mode<T, D, FP4, kSplit>(p, stream);
}

bool rope_append_supported(int dtype, int head_dim) {
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
