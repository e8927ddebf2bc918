// chunk_sched.cuh -- the schedule of attention of several new tokens, the last
// step of a row, and what else its kernels share.
//
// The query rows of a (sequence, kv head) are numbered token by token, the G
// heads of the group beside one another: row n is head n % G of token n / G.
// An item is R consecutive rows of them (the last may have fewer) with the
// tiles of KT cache positions that its tokens attend to.  Laid end to end,
// sequence by sequence, head by head and item by item, the tiles of all items
// form one index space [0, total); CTA w of W takes the slice [w*total/W,
// (w+1)*total/W), the same number of tiles whatever the mix of lengths.
//
// An item cut by slice ends is shared by consecutive CTAs.  Each publishes the
// softmax state of its share (per row the running maximum, the running sum
// and the weighted sum of V: what the per-block aggregation of "KV Cache
// paging in LLM inference", intelliparadigm.com, s2.2, carries from block to
// block) as a record, slot 0 if the share ends the slice's first item, slot 1
// if it begins an item that goes on in the next slice; and CTA w writes
// cuts[w]: which item its slice begins inside of, if that item's first tile
// belongs to the slice before, and the last CTA that shares it.  The second
// launch joins them, and zeroes the rows of sequences whose positions are out of
// range, where nothing waits for it.  No CTA waits for another.  In a record 4 neighbouring
// columns of neighbouring rows lie side by side, so that a row to a thread is
// written and read in whole lines.
//
// The counts and positions are on the device, so every CTA builds the sums over
// sequences itself.  How many tiles the first items of a sequence have is in
// closed form a sum of floor((a i + b) / m).
#pragma once

#include "pa_chunk.h"
#include "pa_device.cuh"

namespace pa {
namespace chunk {

constexpr int kGroups = 1024;              // sums over sequences kept in shared memory
constexpr int kWarpSeqs = 128;             // sequences that a warp sums by itself

// One item and the share [k0, k1) of its tiles that this CTA takes.
struct Item {
    int b, hk, i;              // sequence, kv head, item of the head
    int pos, cnt, nq;          // of the sequence: position of its first new token, new tokens, items per head
    int lo, n;                 // first tile of cache positions, tiles
    int k0, k1;
};

// 16 bytes to shared memory, asynchronously (cp.async groups); zeros unless `take`.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}

// Two fused products and sums in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// New tokens of sequence b and where they start; 0 when there is nothing to do
// or an argument is out of range (*error: the PA_DEVERR bit).
__device__ __forceinline__ int seq_of(const ChunkParams &p, int b, int *pos, int *error) {
    const int cnt = p.counts != nullptr ? __ldg(p.counts + b) : p.T;
    *pos = __ldg(p.positions + b);
    *error = 0;
    if (cnt < 0 || cnt > p.T) {
        *error = PA_DEVERR_BAD_LEN;
        return 0;
    }
    if (*pos < 0 || (int64_t)*pos + cnt > (int64_t)p.MB * p.bs) {
        *error = PA_DEVERR_BAD_POS;
        return 0;
    }
    return cnt;
}

// a / b: a 64-bit quotient costs some hundred cycles, and these are almost
// always small.  Not inlined: what a launch spends on its schedule is for the most
// part instructions that are fetched for the first time.
static __device__ __noinline__ uint64_t quotient(uint64_t a, uint64_t b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// n / G for n < 2^31: with l = ceil(log2 G), the product with ceil(2^(31 + l) / G),
// shifted right by 31 + l (Granlund and Montgomery, "Division by invariant integers
// using multiplication", theorem 4.2).
__device__ __forceinline__ uint32_t by_group(const ChunkParams &p, uint32_t n) {
    return p.g_shift == 0 ? n : __umulhi(n, p.g_mul) >> (p.g_shift - 1);
}

// sum over i < n of floor((a i + b) / m)
__device__ __forceinline__ int64_t floor_sum(uint64_t n, uint64_t m, uint64_t a, uint64_t b) {
    uint64_t s = 0;
    for (;;) {
        if (a >= m) {
            const uint64_t q = quotient(a, m);
            s += (n * (n - 1) / 2) * q;
            a -= q * m;
        }
        if (b >= m) {
            const uint64_t q = quotient(b, m);
            s += n * q;
            b -= q * m;
        }
        const uint64_t y = a * n + b;
        if (y < m) return (int64_t)s;
        n = quotient(y, m);
        b = y - n * m;
        const uint64_t t = m;
        m = a;
        a = t;
    }
}

// Slices: the working CTAs of the grid, no more than there are tiles; CTA w's
// begins at floor(w total / W) = w q + floor(w r / W) with total = q W + r.
struct Slices {
    int64_t total, q;
    int W, r;
    __device__ __forceinline__ void divide(int64_t tiles, int grid) {
        total = tiles;
        W = (int)min((int64_t)grid, total);
        q = W > 0 ? (int64_t)quotient(total, W) : 0;
        r = (int)(total - q * W);
    }
    __device__ __forceinline__ int64_t begin(int w) const { return w * q + (uint32_t)(w * r) / (uint32_t)W; }
    __device__ __forceinline__ int owner(int64_t t) const { return (int)quotient((t + 1) * W - 1, total); }
};

template <int R, int KT>
struct Sched {
    // tiles of item i
    static __device__ __forceinline__ int tiles(const ChunkParams &p, int pos, int cnt, int i, int *lo) {
        const uint32_t rows = (uint32_t)cnt * (uint32_t)p.G, r0 = (uint32_t)i * R;
        const uint32_t last = min(r0 + (uint32_t)R, rows) - 1;
        const int hi = (int)((uint32_t)pos + by_group(p, last)) / KT;
        *lo = p.window > 0 ? max(0, pos + (int)by_group(p, r0) - p.window + 1) / KT : 0;
        return hi - *lo + 1;
    }
    static __device__ __forceinline__ int items(const ChunkParams &p, int cnt) {
        return (int)(((int64_t)cnt * p.G + R - 1) / R);
    }
    // tiles of the first n items of the nq of a head
    static __device__ __noinline__ int64_t tiles_before(const ChunkParams &p, int pos, int cnt, int nq, int n) {
        int64_t s = 0;
        int lo;
        if (n <= 4) {
            for (int i = 0; i < n; ++i) s += tiles(p, pos, cnt, i, &lo);
            return s;
        }
        if (n == nq) s += tiles(p, pos, cnt, --n, &lo);   // the last may have fewer rows
        const uint64_t m = (uint64_t)p.G * KT;
        s += n + floor_sum(n, m, R, (uint64_t)pos * p.G + (R - 1));
        if (p.window > 0) {
            // items whose first token's window begins past position 0
            const int64_t b = ((int64_t)pos - p.window + 1) * p.G;
            const int64_t skip = b >= 0 ? 0 : (-b + R - 1) / R;
            if (skip < n) s -= floor_sum(n - skip, m, R, skip * R + b);
        }
        return s;
    }

    // tiles of sequence b; its error is added to *errors
    static __device__ __forceinline__ int64_t seq_tiles(const ChunkParams &p, int b, int *errors) {
        int pos, error;
        const int cnt = seq_of(p, b, &pos, &error), nq = items(p, cnt);
        *errors |= error;
        return cnt > 0 ? p.Hkv * tiles_before(p, pos, cnt, nq, nq) : 0;
    }

    int64_t at, end;           // tile of the current share's first tile, end of the slice
    Item x;
    int64_t first;             // the current item's first tile

    // Sums over groups of sequences; pre: [kGroups + 1] in shared memory.  Threads
    // 0 to n - 1 (whole warps) call it, with a named barrier of their own; it ends
    // with that barrier.  Returns the sequences of a group.  *errors: of all sequences,
    // though of positions alone (others are reported here).
    static __device__ __forceinline__ int build(const ChunkParams &p, int64_t *pre, int tid, int n, int barrier, int *errors) {
        const int per = (p.B + kGroups - 1) / kGroups, groups = (p.B + per - 1) / per;
        auto sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(n) : "memory"); };
        int mine = 0;
        for (int g = tid; g < groups; g += n) {
            int64_t s = 0;
            for (int b = g * per; b < min(p.B, (g + 1) * per); ++b) s += seq_tiles(p, b, &mine);
            pre[g + 1] = s;
        }
        if (mine != 0 && blockIdx.x == 0) report(p.err_word, mine);
        asm volatile(
            "{\n\t.reg .pred mine, any;\n\tsetp.ne.u32 mine, %3, 0;\n\tbar.red.or.pred any, %1, %2, mine;\n\t"
            "selp.s32 %0, %4, 0, any;\n\t}"
            : "=r"(*errors)
            : "r"(barrier), "r"(n), "r"(mine & PA_DEVERR_BAD_POS), "n"(PA_DEVERR_BAD_POS)
            : "memory");
        if (tid < 32) {                            // inclusive sums, 32 at a time
            int64_t run = 0;
            for (int g0 = 0; g0 < groups; g0 += 32) {
                const int g = g0 + tid;
                int64_t v = g < groups ? pre[g + 1] : 0;
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
                    if (tid >= o) v += y;
                }
                if (g < groups) pre[g + 1] = run + v;
                run += __shfl_sync(0xffffffffu, v, 31);
            }
            if (tid == 0) pre[0] = 0;
        }
        sync();
        return per;
    }

    __device__ __forceinline__ void load_seq(const ChunkParams &p, int b) {
        int error;
        x.b = b;
        x.cnt = seq_of(p, b, &x.pos, &error);
        x.nq = x.cnt > 0 ? items(p, x.cnt) : 0;
    }
    __device__ __forceinline__ void share(const ChunkParams &p) {
        x.n = tiles(p, x.pos, x.cnt, x.i, &x.lo);
        x.k0 = (int)(at - first);
        x.k1 = (int)min((int64_t)x.n, end - first);
    }
    // The first share of this CTA's slice; false when it has none.  Whole warps call
    // it, and any number of them come to the same.
    //
    // Up to kWarpSeqs sequences a warp sums over by itself, without barriers: what a
    // call spends before its first copy is a chain of loads and of instructions
    // fetched for the first time (32 tokens behind 2047 cached ones each: 7 us).
    // More have been summed by build().  *errors: of the lane's sequences.
    __device__ __forceinline__ bool locate(const ChunkParams &p, Slices &sl, int *errors) {
        const int lane = threadIdx.x & 31, per = (p.B + 31) / 32;
        int64_t mine = 0;
        *errors = 0;
        for (int b = lane * per; b < min(p.B, (lane + 1) * per); ++b) mine += seq_tiles(p, b, errors);
        int64_t incl = mine;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        sl.divide(__shfl_sync(0xffffffffu, incl, 31), gridDim.x);
        if ((int)blockIdx.x >= sl.W) return false;
        at = sl.begin(blockIdx.x);
        end = sl.begin(blockIdx.x + 1);
        const int l = __ffs(__ballot_sync(0xffffffffu, incl > at)) - 1;
        enter(p, l * per, at - __shfl_sync(0xffffffffu, incl - mine, l));
        return true;
    }
    __device__ __forceinline__ bool locate(const ChunkParams &p, Slices &sl, const int64_t *pre, int per) {
        const int groups = (p.B + per - 1) / per;
        sl.divide(pre[groups], gridDim.x);
        if ((int)blockIdx.x >= sl.W) return false;
        at = sl.begin(blockIdx.x);
        end = sl.begin(blockIdx.x + 1);
        int lo = 0, hi = groups;                   // pre[lo] <= at < pre[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= at) lo = mid;
            else hi = mid;
        }
        enter(p, lo * per, at - pre[lo]);
        return true;
    }

    // The share at tile `off` of those of sequences b and on.
    __device__ __forceinline__ void enter(const ChunkParams &p, int b, int64_t off) {
        int64_t head = 0;
        for (;; ++b) {
            load_seq(p, b);
            if (x.cnt == 0) continue;
            head = tiles_before(p, x.pos, x.cnt, x.nq, x.nq);
            if (off < head * p.Hkv) break;
            off -= head * p.Hkv;
        }
        x.hk = (int)quotient(off, head);
        off -= x.hk * head;
        // items 32 at a time, a lane each; past many of them, from where the sums lead
        int i0 = 0;
        int64_t before = 0;
        for (int step = 1 << 30; x.nq > 256 && step >= 64; step >>= 1) {
            if (i0 + step >= x.nq) continue;
            const int64_t v = tiles_before(p, x.pos, x.cnt, x.nq, i0 + step);
            if (v <= off) i0 += step, before = v;
        }
        const int lane = threadIdx.x & 31;
        for (;; i0 += 32) {
            int first_tile;
            const int n = i0 + lane < x.nq ? tiles(p, x.pos, x.cnt, i0 + lane, &first_tile) : 0;
            int incl = n;
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            // the first lane whose items reach past off
            const uint32_t past = __ballot_sync(0xffffffffu, before + incl > off);
            if (past != 0) {
                const int l = __ffs(past) - 1;
                before += __shfl_sync(0xffffffffu, incl - n, l);
                i0 += l;
                break;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
        x.i = i0;
        first = at - (off - before);
        share(p);
    }
    // The next share of the slice; false at its end.
    __device__ __forceinline__ bool next(const ChunkParams &p) {
        at = first + x.n;
        if (at >= end) return false;
        first = at;
        if (++x.i == x.nq) {
            x.i = 0;
            if (++x.hk == p.Hkv) {
                x.hk = 0;
                do load_seq(p, x.b + 1);
                while (x.cnt == 0);
            }
        }
        share(p);
        return true;
    }
    __device__ __forceinline__ bool cut() const { return x.k0 > 0 || x.k1 < x.n; }
};

// This CTA's entry of the cuts, from the first share of its slice (has: it has
// one) and the errors of the sequences.
template <int R, int KT>
__device__ __forceinline__ ChunkCut cut_entry(const ChunkParams &p, const Sched<R, KT> &s, bool has, const Slices &sl, int errors) {
    ChunkCut c{};
    c.b = -1;
    c.zeros = (errors & PA_DEVERR_BAD_POS) != 0;
    if (!has || s.x.k0 == 0 || s.first < sl.begin((int)blockIdx.x - 1)) return c;
    c.b = s.x.b;
    c.hk = s.x.hk;
    c.n0 = s.x.i * R;
    c.rows = min(R, s.x.cnt * p.G - c.n0);
    c.last = sl.owner(s.first + s.x.n - 1);
    return c;
}

// Columns c to c + 3 of a row of a record (of `rows` rows in all).
__device__ __forceinline__ float *record_at(float *rec, int rows, int row, int c) { return rec + ((c >> 2) * rows + row) * 4 + (c & 3); }

// The errors that the lanes of a warp found in their sequences, put together and
// reported by CTA 0.
__device__ __forceinline__ int all_errors(const ChunkParams &p, int errors) {
    errors = (int)__reduce_or_sync(0xffffffffu, (unsigned)errors);
    if (errors != 0 && blockIdx.x == 0 && (threadIdx.x & 31) == 0) report(p.err_word, errors);
    return errors;
}

// Byte offset in the pools of the row that holds cache position t of kv head
// hk of sequence b, or -1 when its table entry is out of range.
__device__ __forceinline__ int64_t row_offset(const ChunkParams &p, int b, int hk, int t, int row_bytes) {
    const int j = p.bs_shift >= 0 ? t >> p.bs_shift : t / p.bs;
    const int32_t blk = __ldg(p.block_table + (int64_t)b * p.MB + j);
    if (blk < 0 || blk >= p.num_blocks) return -1;
    return blk * p.block_stride_bytes + ((int64_t)hk * p.bs + (t - j * p.bs)) * row_bytes;
}

// The last step of a row, by one warp: lane l has elements l*N .. l*N + N - 1
// (N = D / 32, or one element for the first D lanes) of the first map's
// weighted sum in o, already divided by its sum, and of the second map's in o2
// (differential form; null: the difference is taken already).  A row that
// attended to a bad block is zeros.
template <typename T, int D, bool DIFF>
__device__ __forceinline__ void finish_row(const ChunkParams &p, const float *o, const float *o2, bool bad, int64_t token,
                                           int head) {
    constexpr int N = D >= 32 ? D / 32 : 1;
    const int lane = threadIdx.x & 31;
    float y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = o[i];
    if constexpr (DIFF) {
        const float lam = __ldg(p.lambdas + head);
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (o2 != nullptr) y[i] -= lam * o2[i];
            sq += y[i] * y[i];
        }
        if (p.norm_weight != nullptr) {
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, s);
            const float r = 1.f / sqrtf(sq * (1.f / D) + p.eps);
            const T *w = reinterpret_cast<const T *>(p.norm_weight) + lane * N;
#pragma unroll
            for (int i = 0; i < N; ++i) y[i] = y[i] * r * Elem<T>::to_float(w[i]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] *= p.out_scale;
    }
    T *dst = reinterpret_cast<T *>(p.out) + (token * p.H + head) * D + lane * N;
    if (D >= 32 || lane < D) {
#pragma unroll
        for (int i = 0; i < N; ++i) dst[i] = Elem<T>::from_float(bad ? 0.f : y[i]);
    }
}

}  // namespace chunk
}  // namespace pa
