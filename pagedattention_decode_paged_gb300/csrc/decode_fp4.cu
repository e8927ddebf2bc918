// decode_fp4.cu -- decode attention over the 4-bit cache (E2M1 codes, one E4M3
// scale per 16 values; include/pagedattn_fp4.h) on the tensor cores.
//
// The per-block attention decomposition is that of "KV Cache paging in LLM
// inference" (intelliparadigm.com) s2.2.  An item is a (sequence, kv head,
// group of query heads); its 32-token tiles are read once for all its heads.
//
// Arithmetic of a tile (one warp, two halves of 16 tokens, mma.sync m16n8k16,
// fp32 accumulation):
//   S^T[16 tokens x 8 columns] = K Q^T, then the online softmax down each
//   column, then O^T[D x 8 columns] += V^T P^T, a column being a query head
//   (16-bit queries) or the high or low fp16 part of one (fp32 queries: the
//   parts' products add up to 22 bits).  One cvt turns two E2M1 codes into
//   fp16, one packed multiply applies the E4M3 scale, exactly; so 4-bit rows
//   go from the ring into MMA A fragments with no staging and no rounding.
//   The contraction over head_dim may take its elements in any order: lane
//   (gid, tig) holds D/8 consecutive bytes of K rows tau(gid), tau(gid) + 8,
//   and the queries are packed to match.  The contraction over tokens needs
//   pairs of tokens side by side: two words of two tokens become the words of
//   their even and odd elements with one shift and one select each, and the
//   cvt then yields (token, next token) pairs.  tau is a permutation of 0..7
//   chosen so that the wide K loads and the V loads both miss no bank.
//   A column's weights are taken against a reference 2^7 below its largest
//   score, and rescaled only when a score passes the reference by more than
//   2^15, so that a tile usually costs one vote and no shuffles.  Inside fp16
//   that leaves the most room below the largest weight: 11 bits down to 2^-21
//   of it, 2^-32 of it below.
//
//   The weights of 16-bit queries are rounded to fp16 for the second product, and
//   not for their sum: f16 outputs of the ragged batch below are 2.6e-4 from the
//   definition, of which their own rounding is 2.1e-4; with two parts for them too
//   they were no further than that, and took 52.9 us for 47.7, 114.5 for 101.5 on
//   64 long sequences.
//
// What bounds it: 4.5 bits per value are so few that a tile's conversions (570
// instructions for 4.6 KB at head_dim 128, half of them on the pipe of the
// integer and conversion instructions) take nearly as long as its bytes.  64
// sequences of 7000 to 8192 tokens, 64 heads on 8, bf16: 102 us where the bytes
// take 83 us at the copy rate, the tile loop itself 88 us; with 16-token tiles 121
// us.  What is left is what a launch costs beside its tiles: lengths, table entries
// and first tiles one after another (6 us until the first tile is multiplied), the
// merge of a CTA's warps (2 us) and, if items are cut between CTAs, of the CTAs (3 to
// 5 us).  32 x 2048 tokens: 23.1 us (bytes 11.3); 256 sequences of 4 to 4096 tokens,
// 32 heads each, f16: 47.7 us (24.8); one of 131071: 35.8 us (22.3).
//
// Work split: the tiles of all items, end to end, are cut into about equal runs,
// one per CTA, and each into equal parts, one per warp (Fp4Cursor, Fp4Runs).  A
// warp that covers an item writes its output; partial states of the warps of
// a CTA meet in shared memory, those of CTAs in the workspace, where the last
// to arrive merges (in two levels when many share an item), always in the
// items' order, so that results repeat.
#include <float.h>
#include <math.h>

#include "balanced.cuh"
#include "fp4.cuh"
#include "pa_rope_fp4.h"

namespace pa {

constexpr int kFp4Tile = 32;       // tokens of a tile: two halves of 16, the MMAs' token axis
constexpr int kFp4Halves = kFp4Tile / 16;
constexpr float kFp4Below = 7.f, kFp4Over = 15.f;   // log2 of a column's largest weight when it is rescaled, and before it is
constexpr float kFp4Empty = -3.402823466e38f;   // reference of a column without scores: below any, and finite
// The rules of the split, each with what the other side of it took:
// - what an item costs beside its tiles (queries, output), in tiles.  256 ragged
//   sequences of 4 to 4096 tokens, median 87: f16, 32 heads of 128 65.6 us at 0, 47.7
//   at 1, 52.7 at 2; 16 heads of 256 (bf16) 65.6, 47.2 and 50.6, of 128 (fp32) 41.0,
//   30.6 and 33.3; but 32 heads of 64 (f16; fp32) 54.1, 38.4 and 37.4; 56.5, 40.3 and
//   38.4, 16 query heads to a kv head of 64 (f16) 29.2, 21.2 and 19.6, 8 to one of 256
//   (bf16) 47.7, 38.3 and 34.9.  One figure for all is within 10% of the best.
constexpr int kFp4Item = 1;
// - tiles per warp below which fewer CTAs share the work.  4 sequences of up to 128
//   tokens: 7.0 us at 1, 7.7 at 2, 9.5 at 4; 4 of 2048: 13.2, 14.1, 14.2 us.
constexpr int kFp4MinTiles = 1;
// - tiles per warp that a CTA may have above the mean to end where items end.  32 x
//   2048 tokens: 25.1 us at 0 (items are cut), 23.1 at 2 to 8; the ragged batch:
//   50.4 at 0 to 3, 47.5 at 4 to 8.
constexpr int kFp4Snap = 4;
// - sharers of an item up to which one level of merging serves (at most 32).  19 CTAs
//   to an item: 37.6 us in two levels, 35.9 in one.
constexpr int kFp4Flat = 24;
// - sharers per first-level group above that.  152 CTAs to an item: 17.3 us with 10,
//   12 or 16.
constexpr int kFp4Group = 12;
constexpr int kFp4Groups = 16;     // such groups: the largest grid has kFp4Groups * kFp4Group CTAs

template <typename T, int D, int NT>
struct Fp4Cfg {
    static constexpr int kParts = sizeof(T) == 4 ? 2 : 1;
    static constexpr int kHeads = NT * 8 / kParts;          // query heads per item
    static constexpr int kRow = D / 2;                      // code bytes of a row
    static constexpr int kScRow = D / 16;                   // scale bytes of a row
    static constexpr int kCodes = 16 * kRow;                // K (or V) codes of a half tile
    static constexpr int kScales = 16 * kScRow;
    static constexpr int kHalf = 2 * (kCodes + kScales);    // K codes, V codes, K scales, V scales
    static constexpr int kStage = kFp4Halves * kHalf;
    static constexpr int kStages = 2;                       // a third changes nothing, and takes room from the schedule
    static constexpr int kWarpRing = kStages * kStage;
    static constexpr int kRec = kHeads * D + 2 * kHeads;    // O, then m, then l
    // one CTA per SM: of 12 warps where a thread gets along with 168 registers (8
    // warps: 58.9 us where 12 take 47.6 on the ragged batch, 25.0 and 23.3 on 32 x 2048;
    // the 16-bit kernels of head_dim 64 with two column tiles spill 8 bytes)
    static constexpr int kWarps = NT * D <= 128 ? 12 : 8;
    static constexpr int kThreads = kWarps * 32;
    // the last record of a warp takes the place of its ring
    static constexpr int kRingBytes = kWarpRing > kRec * 4 ? kWarpRing : kRec * 4;
    static_assert(kRec <= kFp4RecFloats, "a record fits the workspace");
    static constexpr size_t kFixed = (size_t)kWarps * (kRingBytes + kRec * 4);
    static constexpr int kMost = kFixed / (kRec * 4) < 32 ? (int)(kFixed / (kRec * 4)) : 32;   // records merged at once
    static constexpr int kFlat = kFp4Flat < kMost ? kFp4Flat : kMost;
    static_assert(kMost >= kFp4Group && kMost >= kFp4Groups, "the records of either level fit");
    static_assert(kRec % 4 == 0 && kFp4RecFloats % 4 == 0, "records are whole 16-byte pieces");
    static size_t bytes(int batch) { return kFixed + ((size_t)2 * batch + 1) * 4; }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src) {
    if constexpr (N == 16) cp_async16(dst, src);
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Tiles of a sequence of L tokens.
__device__ __forceinline__ int32_t fp4_window_start(int32_t L, int32_t window) {
    return window > 0 && L > window ? L - window : 0;
}
__device__ __forceinline__ int32_t fp4_tiles(int32_t L, int32_t window) {
    return (L - fp4_window_start(L, window) / kFp4Tile * kFp4Tile + kFp4Tile - 1) / kFp4Tile;
}

// W equal runs of T places: run w starts at floor(w T / W).  With T = q W + r
// that is w q + floor(w r / W), and w r + 1/2 over W is further from an integer
// than fp32 rounds it for every W up to 1024, so no division is needed.
struct Fp4Runs {
    int32_t T, W, q, r;
    float inv;
    __device__ __forceinline__ Fp4Runs(int32_t places, int32_t runs)
        : T(places), W(runs), q(places / runs), r(places % runs), inv(1.f / (float)runs) {}
    __device__ __forceinline__ int32_t start(int32_t w) const { return w * q + (int32_t)(((float)(w * r) + 0.5f) * inv); }
    __device__ __forceinline__ int32_t owner(int32_t t) const {   // of place t
        int32_t w = min(W - 1, (int32_t)(((float)t + 0.5f) * ((float)W / (float)T)));
        while (w > 0 && start(w) > t) --w;
        while (w + 1 < W && start(w + 1) <= t) ++w;
        return w;
    }
};

// A place in the index space of the work: an item of n tiles covers kFp4Item +
// n places from `first` on, its tiles the last n.
struct Fp4Cursor {
    int b, it, n;
    int32_t first;

    __device__ __forceinline__ void seek(const int32_t *pre, const int32_t *lens, int32_t window, int B, int32_t t) {
        int lo = 0, hi = B;                    // pre[lo] <= t < pre[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= t) lo = mid;
            else hi = mid;
        }
        b = lo;
        n = fp4_tiles(lens[b], window);
        // the quotient is below 2^20, so that in fp32 it is off by one at most
        const int32_t places = n + kFp4Item, at = t - pre[b];
        it = (int32_t)__fdividef((float)at, (float)places);
        if (it * places > at) --it;
        else if ((it + 1) * places <= at) ++it;
        first = pre[b] + it * places;
    }
    // To the next item; b is B behind the last one.
    __device__ __forceinline__ void next(const int32_t *pre, const int32_t *lens, int32_t window, int B, int items_per_seq) {
        first += n + kFp4Item;
        if (++it < items_per_seq) return;
        it = 0;
        do {
            ++b;
        } while (b < B && pre[b + 1] == pre[b]);
        if (b < B) n = fp4_tiles(lens[b], window);
    }
};

// The schedule in shared memory: pre[b] the first place of sequence b, pre[B]
// their number, lens[b] the length (-1: invalid).  Sequences with nothing to
// attend to have no places.
__device__ __forceinline__ void fp4_schedule(const DecodeParams &p, int items_per_seq, int32_t *pre, int32_t *lens,
                                             int32_t *scan_tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    int32_t s = 0;
    for (int b = b0; b < b1; ++b) {
        const int32_t L = p.seq_lens[b];
        const bool ok = L >= 0 && (int64_t)L <= (int64_t)p.MB * p.bs;
        const int32_t n = ok ? fp4_tiles(L, p.window) : 0;
        lens[b] = ok ? L : -1;
        pre[b] = n > 0 ? (n + kFp4Item) * items_per_seq : 0;
        s += pre[b];
        if (!ok && (int)(b % gridDim.x) == (int)blockIdx.x) report(p.err_word, PA_DEVERR_BAD_LEN);
    }
    int32_t incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scan_tmp[warp] = incl;
    __syncthreads();
    int32_t run = incl - s;
    for (int w = 0; w < warp; ++w) run += scan_tmp[w];
    for (int b = b0; b < b1; ++b) {
        const int32_t c = pre[b];
        pre[b] = run;
        run += c;
    }
    if (threadIdx.x == blockDim.x - 1) pre[p.B] = run;
    __syncthreads();
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ float4 lds_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// Row of the tile behind row i of the MMAs' token axis (rows 8..15: + 8), and
// where 16-byte chunk c of tile row r lies in its row.
template <int D>
__device__ __forceinline__ int tau(int i) {
    return D == 64 ? i ^ ((i >> 2) & 1) : i ^ ((i >> 1) & 1);
}
template <int D>
__device__ __forceinline__ int swizzle(int r, int c) {
    return D == 64 ? c : D == 128 ? c ^ ((r >> 1) & 3) : c ^ (r & 7);
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t *w) {
    if constexpr (N == 1) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
    if constexpr (N == 2) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}
template <int BYTES>
__device__ __forceinline__ uint32_t lds_bytes(uint32_t addr) {
    uint32_t v;
    if constexpr (BYTES == 1) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    else if constexpr (BYTES == 2) asm volatile("{\n\t.reg .u16 t;\n\tld.shared.u16 t, [%1];\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(v) : "r"(addr));
    else asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// WHOLE: block_size is a multiple of 16, so the 16 rows of half a tile are
// contiguous and one table entry serves them; else every row is looked up by
// itself (32 x 2048 in blocks of 16: 27.3 us so, 23.3 whole).  Either way a tile is
// a 16-byte asynchronous copy per lane and chunk.
template <typename T, int D, int NT, bool WHOLE>
__global__ void __launch_bounds__((Fp4Cfg<T, D, NT>::kThreads), 1)
decode_fp4_kernel(const __grid_constant__ Fp4Decode fp, const int units_per_kv) {
    using C = Fp4Cfg<T, D, NT>;
    constexpr int P = C::kParts, HP = C::kHeads, S = C::kStages, W = C::kWarps;
    constexpr int KW = D / 32;                 // words of a K row per lane
    constexpr int VW = D / 64;                 // words of a V row per lane
    constexpr int MT = D / 16;                 // 16-row tiles of O^T
    const DecodeParams &p = fp.d;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ int32_t scan_tmp[W];
    __shared__ int32_t rec_first[2 * W], rec_n[2 * W], rec_b[2 * W], rec_it[2 * W];
    __shared__ int32_t arrived[2], sharers_of[2];
    __shared__ uint32_t rec_at[32];            // records to merge, in shared memory
    __shared__ const float *source[2][32];     // those of other CTAs, in the workspace
    __shared__ float *merged_to[2];            // null: the output
    __shared__ int32_t snap[kFp4Groups * kFp4Group + 1];
    __shared__ int32_t group_rec[2 * W + 1];   // of the items merged in this CTA: first record, and its place in rec_at

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    unsigned char *ring_p = smem + (size_t)warp * C::kRingBytes;
    const uint32_t ring = smem_u32(ring_p);
    float *first_rec = reinterpret_cast<float *>(smem + (size_t)W * C::kRingBytes) + (size_t)warp * C::kRec;
    float *last_rec = reinterpret_cast<float *>(ring_p);
    int32_t *pre = reinterpret_cast<int32_t *>(smem + C::kFixed);
    int32_t *lens = pre + p.B + 1;

    grid_dependency_wait();
    allow_dependents();
    // the table is on its way to L2 while the lengths are read: a line per thread
    {
        const int64_t line = (int64_t)threadIdx.x * gridDim.x + blockIdx.x;
        if (line * 32 < (int64_t)p.B * p.MB) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.block_table + line * 32));
    }
    const int items_per_seq = p.Hkv * units_per_kv;
    fp4_schedule(p, items_per_seq, pre, lens, scan_tmp);
    zero_empty_sequences<T>(p, pre);
    const int32_t Tn = pre[p.B];
    // An equal run of places to every CTA (fewer CTAs when their warps would have
    // less than kFp4MinTiles).  The runs' ends are moved to the nearest ends of
    // items, and nothing has to be merged between CTAs, if that leaves no CTA
    // with much more than the mean.
    const int nC = min((int)gridDim.x, (Tn + W * kFp4MinTiles - 1) / (W * kFp4MinTiles));
    const int cta = blockIdx.x;
    if (cta >= nC) return;
    const Fp4Runs runs(Tn, nC);
    for (int c = threadIdx.x; c <= nC; c += C::kThreads) {
        int32_t t = runs.start(c);
        if (c > 0 && c < nC) {
            Fp4Cursor x;
            x.seek(pre, lens, p.window, p.B, t);
            t = 2 * (t - x.first) <= x.n + kFp4Item ? x.first : x.first + x.n + kFp4Item;
        }
        snap[c] = t;
    }
    __syncthreads();
    bool over = false;
    for (int c = threadIdx.x; c < nC; c += C::kThreads) over |= snap[c + 1] - snap[c] > runs.q + W * kFp4Snap;
    const bool cut = __syncthreads_or(over);   // items are cut between CTAs
    const int32_t c0 = cut ? runs.start(cta) : snap[cta], c1 = cut ? runs.start(cta + 1) : snap[cta + 1];
    if (c0 >= c1) return;
    const Fp4Runs warp_runs(c1 - c0, W);
    const int32_t w0 = c0 + warp_runs.start(warp), w1 = c0 + warp_runs.start(warp + 1);
    if (lane < 2) rec_first[2 * warp + lane] = -1;

    const int grp = p.H / p.Hkv;               // query heads per kv head
    T *out = reinterpret_cast<T *>(p.out);

    // ---- producer side -------------------------------------------------------
    // Table entries are looked up ahead, so that a tile's copies never wait for
    // them: WHOLE, of a batch of up to 16 tiles of an item, lane i keeping the
    // offsets of the i-th half tile; else of one tile, lane l of its row l.
    Fp4Cursor pc = {};
    int32_t p_k = 0, p_end = 0;                // the batch's first tile, the last of this warp's run of its item
    int p_i = 0, p_left = 0;                   // the next tile in it, tiles left in it
    bool p_more = true;                        // there may be a batch behind it
    int64_t p_code = -1, p_scale = 0;          // byte offsets of K's codes (-1: nothing to fetch) and scales
    uint32_t p_bad = 0;                        // half tiles (rows) whose entry is outside the pool
    uint32_t bad_tiles = 0;                    // bit i: the tile i after the next one had a bad table entry
    const int64_t v_scale_off = (int64_t)p.Hkv * p.bs * C::kScRow;
    auto look_up = [&]() {                     // the batch behind the one that is done
        p_k += p_i;
        p_i = 0;
        if (p_k >= p_end) {
            pc.next(pre, lens, p.window, p.B, items_per_seq);
            p_k = 0;
            p_end = min(pc.n, w1 - pc.first - kFp4Item);
            p_more = pc.b < p.B && p_end > 0;
            if (!p_more) return;
        }
        const int32_t L = lens[pc.b];
        const int32_t t_win = fp4_window_start(L, p.window);
        const int32_t base = t_win / kFp4Tile * kFp4Tile + p_k * kFp4Tile;
        const int hk = units_per_kv == 1 ? pc.it : pc.it / units_per_kv;
        p_left = WHOLE ? min(32 / kFp4Halves, p_end - p_k) : 1;
        // tokens [tok, tok + (WHOLE ? 16 : 1)) of this lane; needed if one of them is attended to
        const int32_t tok = base + lane * (WHOLE ? 16 : 1);
        const bool need = lane < p_left * (WHOLE ? kFp4Halves : kFp4Tile) && tok < L && tok + (WHOLE ? 16 : 1) > t_win;
        int64_t blk = 0;
        int slot = 0;
        if (need) {
            const int32_t j = p.bs_shift >= 0 ? tok >> p.bs_shift : tok / p.bs;
            slot = tok - j * p.bs;
            blk = __ldg(p.block_table + (int64_t)pc.b * p.MB + j);
        }
        const bool bad = blk < 0 || blk >= p.num_blocks;
        if (bad) report(p.err_word, PA_DEVERR_BAD_BLOCK);
        p_bad = __ballot_sync(0xffffffffu, bad);
        const int64_t row = (int64_t)hk * p.bs + slot;
        p_code = need && !bad ? blk * p.block_stride_bytes + row * C::kRow : -1;
        p_scale = (blk * 2 * p.Hkv * p.bs + row) * C::kScRow;
        if (p_k == 0) {                        // the item's queries, before its first tile is due
            const char *q = reinterpret_cast<const char *>(p.q) +
                            ((int64_t)pc.b * p.H + hk * grp + (pc.it - hk * units_per_kv) * HP) * D * sizeof(T);
            const int heads = min(HP, grp - (pc.it - hk * units_per_kv) * HP);
            for (int i = lane * 128; i < heads * D * (int)sizeof(T); i += 32 * 128)
                asm volatile("prefetch.global.L1 [%0];" ::"l"(q + i));
        }
    };
    constexpr int CH = C::kRow / 16;           // 16-byte chunks per row
    constexpr int RS = 32 / CH;                // rows per copy instruction
    const int f_r = lane / CH, f_c = lane % CH;
    const uint32_t f_dst = f_r * C::kRow + swizzle<D>(f_r, f_c) * 16;
    // RS rows on, the swizzle is the same, but for D 256 (4 rows a copy) its 4s bit
    static_assert(RS % 8 == 0 || (D == 256 && RS == 4), "");
    const uint32_t f_sdst = 2 * C::kCodes + lane * C::kScRow;
    const char *f_k = p.k_pool + f_r * C::kRow + f_c * 16, *f_v = p.v_pool + f_r * C::kRow + f_c * 16;
    const uint8_t *f_s = fp.scales + (lane & 15) * C::kScRow + (lane >> 4) * v_scale_off;
    auto fetch = [&](uint32_t slot) {          // the next tile into the ring
#pragma unroll
        for (int half = 0; half < kFp4Halves; ++half, slot += C::kHalf) {
            if constexpr (WHOLE) {
                const int64_t off = __shfl_sync(0xffffffffu, p_code, p_i * kFp4Halves + half);
                const int64_t so = __shfl_sync(0xffffffffu, p_scale, p_i * kFp4Halves + half);
                if (off < 0) continue;         // nothing there that is attended to, or a bad entry
                cp_async_small<C::kScRow>(slot + f_sdst, f_s + so);
                const char *ks = f_k + off, *vs = f_v + off;
#pragma unroll
                for (int i = 0; i < 16 / RS; ++i) {
                    const uint32_t dst = slot + (D == 256 && (i & 1) ? f_dst ^ 64u : f_dst) + i * RS * C::kRow;
                    cp_async16(dst, ks + i * RS * C::kRow);
                    cp_async16(dst + C::kCodes, vs + i * RS * C::kRow);
                }
            } else {
                const int64_t mine = __shfl_sync(0xffffffffu, p_code, half * 16 + (lane & 15));
                const int64_t so = __shfl_sync(0xffffffffu, p_scale, half * 16 + (lane & 15));
                if (mine >= 0) cp_async_small<C::kScRow>(slot + f_sdst, fp.scales + so + (lane >> 4) * v_scale_off);
#pragma unroll
                for (int i = 0; i < 16 / RS; ++i) {
                    const int r = i * RS + f_r;
                    const int64_t off = __shfl_sync(0xffffffffu, p_code, half * 16 + r);
                    if (off < 0) continue;
                    const uint32_t dst = slot + r * C::kRow + swizzle<D>(r, f_c) * 16;
                    cp_async16(dst, p.k_pool + off + f_c * 16);
                    cp_async16(dst + C::kCodes, p.v_pool + off + f_c * 16);
                }
            }
        }
        if (p_bad != 0 && (!WHOLE || ((p_bad >> (p_i * kFp4Halves)) & ((1u << kFp4Halves) - 1u)) != 0))
            bad_tiles |= 1u << (S - 2);
        ++p_i;
        --p_left;
    };

    // ---- consumer side -------------------------------------------------------
    uint32_t qf[NT][MT][2];                    // Q^T as MMA B fragments
    float cs[NT][2];                           // scale * log2(e) * 2^e of columns 2 tig, 2 tig + 1
    float o[NT][MT][4], m[NT][2], l[NT][2], nm[kFp4Halves][2][NT][2];
    auto load_q = [&](int b, int it) {
        const int hk = it / units_per_kv, h0 = (it - hk * units_per_kv) * HP;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = P == 2 ? nt * 4 + (gid & 3) : nt * 8 + gid;
            const bool have = h0 + col < grp;
            const T *src = reinterpret_cast<const T *>(p.q) + ((int64_t)b * p.H + hk * grp + h0 + col) * D + tig * (D / 4);
            constexpr int VEC = D / 4 * (int)sizeof(T) / 16;
            uint4 raw[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) raw[i] = have ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0, 0, 0, 0);
            constexpr int PER = 16 / (int)sizeof(T);
            float big = 0.f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float x[PER];
                Elem<T>::unpack(raw[i], x);
#pragma unroll
                for (int j = 0; j < PER; ++j) big = fmaxf(big, fabsf(x[j]));
            }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            // a power of two that brings the head's largest element into [2^14, 2^15), as
            // far below fp16's largest value as leaves its parts the most bits; no
            // further than `up` is a normal number
            int e = (int)((__float_as_uint(big) >> 23) & 255u) - 127;
            e = big > 0.f && e < 128 ? max(e, -112) - 14 : 0;
            const float down = __uint_as_float((uint32_t)(127 - e) << 23);
            const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float x[PER];
                Elem<T>::unpack(raw[i], x);
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    x[j] *= down;
                    if (P == 2 && gid >= 4) x[j] -= __half2float(__float2half_rn(x[j]));
                }
#pragma unroll
                for (int j = 0; j < PER / 2; ++j) {
                    const int w = i * (PER / 2) + j;
                    qf[nt][w / 2][w & 1] = Elem<__half>::pack2(x[2 * j], x[2 * j + 1]);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = P == 2 ? (2 * tig + j) & 3 : 2 * tig + j;
                // finite, so that it leaves a product of 0 (masked rows among them) as it is
                cs[nt][j] = fminf(fmaxf(p.scale_log2 * __shfl_sync(0xffffffffu, up, c * 4), -FLT_MAX), FLT_MAX);
                m[nt][j] = kFp4Empty;
                l[nt][j] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][mt][i] = 0.f;
        }
    };

    // Scores are taken relative to the columns' references m: nm[half][r][.] is
    // -m, or -inf if this lane's row r of the half lies outside the item.
    auto tile = [&](uint32_t slot) {
        const int rk = tau<D>(gid);
        float c[kFp4Halves][NT][4];
#pragma unroll
        for (int half = 0; half < kFp4Halves; ++half) {
            const uint32_t codes = slot + half * C::kHalf, sc = codes + 2 * C::kCodes;
            // K rows rk and rk + 8 of this lane, and their scales
            uint32_t kw[2][KW], ks[2][(KW + 1) / 2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = rk + 8 * r;
                if constexpr (D == 256) {
                    lds_words<4>(codes + row * C::kRow + swizzle<D>(row, 2 * tig) * 16, kw[r]);
                    lds_words<4>(codes + row * C::kRow + swizzle<D>(row, 2 * tig + 1) * 16, kw[r] + 4);
                } else {
                    lds_words<KW>(codes + row * C::kRow + (D == 128 ? swizzle<D>(row, tig) * 16 : tig * 8), kw[r]);
                }
                const uint32_t s = lds_bytes<KW / 2>(sc + row * C::kScRow + tig * (KW / 2));
#pragma unroll
                for (int i = 0; i < KW / 2; ++i) ks[r][i] = e4m3x2_to_f16x2(__byte_perm(s, 0, i * 0x11));
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) c[half][nt][i] = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const uint32_t s0 = ks[0][w / 2], s1 = ks[1][w / 2];
                const uint32_t a[4] = {hmul2_u32(e2m1x2_to_f16x2<0>(kw[0][w]), s0), hmul2_u32(e2m1x2_to_f16x2<0>(kw[1][w]), s1),
                                       hmul2_u32(e2m1x2_to_f16x2<1>(kw[0][w]), s0), hmul2_u32(e2m1x2_to_f16x2<1>(kw[1][w]), s1)};
                const uint32_t d[4] = {hmul2_u32(e2m1x2_to_f16x2<2>(kw[0][w]), s0), hmul2_u32(e2m1x2_to_f16x2<2>(kw[1][w]), s1),
                                       hmul2_u32(e2m1x2_to_f16x2<3>(kw[0][w]), s0), hmul2_u32(e2m1x2_to_f16x2<3>(kw[1][w]), s1)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    MmaOp<__half>::run(c[half][nt], a, qf[nt][2 * w][0], qf[nt][2 * w][1]);
                    MmaOp<__half>::run(c[half][nt], d, qf[nt][2 * w + 1][0], qf[nt][2 * w + 1][1]);
                }
            }
        }

        // scores in the log2 domain, relative to the columns' references
        float x[kFp4Halves][NT][4];
        bool over = false;
#pragma unroll
        for (int half = 0; half < kFp4Halves; ++half)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (P == 2) c[half][nt][i] += __shfl_xor_sync(0xffffffffu, c[half][nt][i], 2);
                    x[half][nt][i] = fmaf(c[half][nt][i], cs[nt][i & 1], nm[half][i >> 1][nt][i & 1]);
                    over = over || x[half][nt][i] > kFp4Over;
                }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float y[2 * kFp4Halves], mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 2 * kFp4Halves; ++i) {
                        y[i] = nm[i / 2][i & 1][nt][j] == -INFINITY ? -INFINITY : c[i / 2][nt][(i & 1) * 2 + j] * cs[nt][j];
                        mx = fmaxf(mx, y[i]);
                    }
#pragma unroll
                    for (int s = 4; s < 32; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
                    mx = fmaxf(m[nt][j], mx - kFp4Below);
                    const float f = ex2_approx(m[nt][j] - mx);
                    m[nt][j] = mx;
                    l[nt][j] *= f;
#pragma unroll
                    for (int i = 0; i < 2 * kFp4Halves; ++i) {
                        if (nm[i / 2][i & 1][nt][j] != -INFINITY) nm[i / 2][i & 1][nt][j] = -mx;
                        x[i / 2][nt][(i & 1) * 2 + j] = y[i] - mx;
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        o[nt][mt][j] *= f;
                        o[nt][mt][j + 2] *= f;
                    }
                }
        }
#pragma unroll
        for (int half = 0; half < kFp4Halves; ++half) {
            const uint32_t codes = slot + half * C::kHalf;
            uint32_t pf[NT][2];                // P^T as MMA B fragments
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = ex2_approx(x[half][nt][i]);
                    l[nt][i & 1] += w[i];
                    if (P == 2 && tig >= 2) w[i] -= __half2float(__float2half_rn(w[i]));
                }
                pf[nt][0] = movmatrix_trans(Elem<__half>::pack2(w[0], w[1]));
                pf[nt][1] = movmatrix_trans(Elem<__half>::pack2(w[2], w[3]));
            }

            // V rows of this lane's token pairs (t0, t1) and (t0 + 8, t1 + 8)
            const int t0 = tau<D>(2 * tig), t1 = tau<D>(2 * tig + 1);
            const uint32_t vc = codes + C::kCodes, vs = codes + 2 * C::kCodes + C::kScales;
            uint32_t vw[4][VW], ss[2][(VW + 1) / 2];
            constexpr int VB = VW == 4 ? 2 : 1;    // scale bytes per lane and row
            uint32_t sb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (i & 1 ? t1 : t0) + 8 * (i >> 1);
                const int byte = gid * (D / 16);   // of the row
                lds_words<VW>(vc + row * C::kRow + swizzle<D>(row, byte / 16) * 16 + byte % 16, vw[i]);
                sb[i] = lds_bytes<VB>(vs + row * C::kScRow + (D == 64 ? gid / 2 : gid * VB));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < VB; ++k)
                    ss[i][k] = e4m3x2_to_f16x2(__byte_perm(sb[2 * i], sb[2 * i + 1], k | ((4 + k) << 4)));
#pragma unroll
            for (int v = 0; v < VW; ++v) {
                uint32_t ev[2], od[2];         // even and odd elements of a token pair
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t a = vw[2 * i][v], b = vw[2 * i + 1][v];
                    ev[i] = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
                    od[i] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
                }
                const uint32_t s0 = ss[0][VB == 2 ? v / 2 : 0], s1 = ss[1][VB == 2 ? v / 2 : 0];
                auto step = [&](int j, uint32_t e0, uint32_t d0, uint32_t e1, uint32_t d1) {
                    const uint32_t a[4] = {hmul2_u32(e0, s0), hmul2_u32(d0, s0), hmul2_u32(e1, s1), hmul2_u32(d1, s1)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) MmaOp<__half>::run(o[nt][4 * v + j], a, pf[nt][0], pf[nt][1]);
                };
                step(0, e2m1x2_to_f16x2<0>(ev[0]), e2m1x2_to_f16x2<0>(od[0]), e2m1x2_to_f16x2<0>(ev[1]), e2m1x2_to_f16x2<0>(od[1]));
                step(1, e2m1x2_to_f16x2<1>(ev[0]), e2m1x2_to_f16x2<1>(od[0]), e2m1x2_to_f16x2<1>(ev[1]), e2m1x2_to_f16x2<1>(od[1]));
                step(2, e2m1x2_to_f16x2<2>(ev[0]), e2m1x2_to_f16x2<2>(od[0]), e2m1x2_to_f16x2<2>(ev[1]), e2m1x2_to_f16x2<2>(od[1]));
                step(3, e2m1x2_to_f16x2<3>(ev[0]), e2m1x2_to_f16x2<3>(od[0]), e2m1x2_to_f16x2<3>(ev[1]), e2m1x2_to_f16x2<3>(od[1]));
            }
        }
    };

    // A record's O lies as the lanes hold it, so that no store misses a bank: a
    // slab is four elements of every lane.  Slab i of lane l (two parts: half the
    // slabs each of lanes tig and tig + 2, which hold the same sums) is head
    // head_of(i, l), elements dim_of(i, l)...
    constexpr int SLABS = HP * D / 128;
    auto slab_of = [](int i, int t) { return P == 2 ? i + (t >> 1) * SLABS : i; };   // (nt, j, v, quarter) of lane's i-th
    auto head_of = [&](int i, int ln) {
        const int s = slab_of(i, ln & 3);
        return s / (4 * VW) * (8 / P) + (P == 2 ? 2 * (ln & 1) : 2 * (ln & 3)) + s / (2 * VW) % 2;
    };
    auto dim_of = [&](int i, int ln) {
        const int s = slab_of(i, ln & 3);
        return (ln >> 2) * (D / 8) + s / 2 % VW * 8 + s % 2 * 4;
    };
    // The state of an item this warp has finished its part of: whole items to
    // `out`, parts to a record (O, m [HP], l [HP]; l < 0: bad table).
    auto finish = [&](const Fp4Cursor &cc, bool whole, bool bad, float *rec) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], s);
            }
            if constexpr (P == 2) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[nt][mt][i] += __shfl_xor_sync(0xffffffffu, o[nt][mt][i], 2);
            }
        }
        const int hk = cc.it / units_per_kv, h0 = (cc.it - hk * units_per_kv) * HP;
        const bool writer = P == 1 || tig < 2;
        if (!whole) {
#pragma unroll
            for (int s = 0; s < SLABS * P; ++s) {
                const int nt = s / (4 * VW), j = s / (2 * VW) % 2, mt = s / 2 % VW * 4 + s % 2 * 2;
                const float4 x = make_float4(o[nt][mt][j], o[nt][mt][j + 2], o[nt][mt + 1][j], o[nt][mt + 1][j + 2]);
                if (P == 1 || (tig >> 1) == s / SLABS)
                    *reinterpret_cast<float4 *>(rec + (s % SLABS) * 128 + lane * 4) = x;
            }
            if (gid == 0 && writer)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int col = nt * (8 / P) + 2 * tig + j;
                        rec[HP * D + col] = m[nt][j];
                        rec[HP * D + HP + col] = bad ? -1.f : l[nt][j];
                    }
            return;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = nt * (8 / P) + 2 * tig + j;
                if (!writer || h0 + col >= grp) continue;
                const float f = fp.v_g / l[nt][j];
#pragma unroll
                for (int v = 0; v < VW; ++v) {
                    float x[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[2 * k] = bad ? 0.f : o[nt][4 * v + k][j] * f;
                        x[2 * k + 1] = bad ? 0.f : o[nt][4 * v + k][j + 2] * f;
                    }
                    store8(out + ((int64_t)cc.b * p.H + hk * grp + h0 + col) * D + gid * (D / 8) + 8 * v, x);
                }
            }
    };

    if (w0 < w1) {
        pc.seek(pre, lens, p.window, p.B, w0);
        Fp4Cursor cc = pc;
        p_k = max(0, w0 - pc.first - kFp4Item);
        p_end = min(pc.n, w1 - pc.first - kFp4Item);
#pragma unroll 1
        for (int i = -1; i < S - 1; ++i) {     // the first batch, and its first tiles
            bad_tiles >>= 1;
            if (p_left > 0) fetch(ring + i * C::kStage);
            if (i >= 0) cp_async_commit();
            if (p_left == 0 && p_more) look_up();
        }
        uint32_t now = ring, free_slot = ring + (S - 1) * C::kStage;   // the tile's slot, that of the tile before
#pragma unroll 1
        for (; cc.b < p.B && cc.first < w1; cc.next(pre, lens, p.window, p.B, items_per_seq)) {
            int32_t k = max(0, w0 - cc.first - kFp4Item);
            const int32_t end = min(cc.n, w1 - cc.first - kFp4Item);
            if (k >= end) continue;
            const bool whole = k == 0 && end == cc.n;
            load_q(cc.b, cc.it);
            const int32_t hi = lens[cc.b], lo = fp4_window_start(hi, p.window);
            // tiles with rows outside the item: its first (of a window) and its last
            const int32_t lo_edge = lo % kFp4Tile != 0 ? 0 : -1, hi_edge = hi % kFp4Tile != 0 ? cc.n - 1 : -1;
            int32_t first_k = k;               // where nm is to be set anew
            bool bad = false;
#pragma unroll 1
            for (; k < end; ++k) {
                cp_async_wait<S - 2>();
                __syncwarp();                  // every lane's copies have landed, and the tile before is read
                if (bad_tiles != 0) {
                    bad |= bad_tiles & 1u;
                    bad_tiles >>= 1;
                }
                if (p_left > 0) fetch(free_slot);
                cp_async_commit();
                if (p_left == 0 && p_more) look_up();
                const bool edge = k == lo_edge || k == hi_edge;
                if (edge || k == first_k) {
                    // rows outside: no weight, and scales of 0, for a slot that nobody
                    // wrote may hold NaN, which no weight would remove
                    const int32_t tok0 = (lo / kFp4Tile + k) * kFp4Tile;
#pragma unroll
                    for (int half = 0; half < kFp4Halves; ++half) {
                        const int32_t r = tok0 + half * 16 + (lane & 15);
                        if (r < lo || r >= hi) {
#pragma unroll
                            for (int i = 0; i < C::kScRow; i += 4)
                                asm volatile("st.shared.b32 [%0], %1;" ::"r"(now + half * C::kHalf + f_sdst + i), "r"(0)
                                             : "memory");
                        }
#pragma unroll
                        for (int row = 0; row < 2; ++row) {
                            const int32_t rr = tok0 + half * 16 + tau<D>(gid) + 8 * row;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int j = 0; j < 2; ++j) nm[half][row][nt][j] = rr < lo || rr >= hi ? -INFINITY : -m[nt][j];
                        }
                    }
                    __syncwarp();
                }
                tile(now);
                if (k == lo_edge) first_k = k + 1;   // the rows are inside again
                free_slot = now;
                now = now + C::kStage == ring + S * C::kStage ? ring : now + C::kStage;
            }
            if (end < cc.n) {                  // the last part of the run: the ring is free for its record
                cp_async_wait<0>();
                __syncwarp();
            }
            finish(cc, whole, bad, end < cc.n ? last_rec : first_rec);
            if (!whole && lane == 0) {
                const int r = 2 * warp + (end < cc.n ? 1 : 0);
                rec_first[r] = cc.first;
                rec_n[r] = cc.n;
                rec_b[r] = cc.b;
                rec_it[r] = cc.it;
            }
        }
    }
    __syncthreads();

    // ---- merges --------------------------------------------------------------
    // Element i (a lane's slab) of the records rec_at[from, to) of one item, merged
    // into its output, or into the record dst.  One copy of this code serves every
    // merge, and a short one: what a CTA runs once is paid for in instruction fetches
    // (8 records at a time: 47.8 us for 47.4 on the ragged batch, 36.1 for 35.9 on 1 x
    // 131071).
    constexpr int kBatch = 4;                  // records loaded at a time
    const int elements = (grp == 1 && NT == 1 && P == 1 ? SLABS / 2 : SLABS) * 32;   // one head: the slabs of j = 0
    auto merge = [&](int from, int to, int b, int it, float *dst, int i) {
        const int hk = it / units_per_kv, h0 = (it - hk * units_per_kv) * HP;
        const int ln = i & 31, h = head_of(i >> 5, ln), d = dim_of(i >> 5, ln);
        float M = kFp4Empty, sum = 0.f;
        bool bad = false;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int r = from; r < to; r += kBatch) {
            uint32_t rec[kBatch];
            float mr[kBatch], lr[kBatch];
            float4 a[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) rec[k] = rec_at[min(r + k, to - 1)];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                mr[k] = lds_f32(rec[k] + (HP * D + h) * 4);
                lr[k] = lds_f32(rec[k] + (HP * D + HP + h) * 4);
                a[k] = lds_f32x4(rec[k] + i * 16);
            }
            float top = M;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) top = fmaxf(top, mr[k]);
            const float f = ex2_approx(M - top);
            M = top;
            sum *= f;
            acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (r + k < to) {
                    const float w = ex2_approx(mr[k] - top);
                    bad |= lr[k] < 0.f;
                    sum = fmaf(lr[k], w, sum);
                    acc.x = fmaf(a[k].x, w, acc.x);
                    acc.y = fmaf(a[k].y, w, acc.y);
                    acc.z = fmaf(a[k].z, w, acc.z);
                    acc.w = fmaf(a[k].w, w, acc.w);
                }
        }
        if (dst != nullptr) {
            *reinterpret_cast<float4 *>(dst + i * 4) = acc;
            if (d == 0) {
                dst[HP * D + h] = M;
                dst[HP * D + HP + h] = bad ? -1.f : sum;
            }
        } else if (h0 + h < grp) {
            const float f = fp.v_g / sum;
            T *o4 = out + ((int64_t)b * p.H + hk * grp + h0 + h) * D + d;
            const float4 y = bad ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
            if constexpr (sizeof(T) == 4) *reinterpret_cast<float4 *>(o4) = y;
            else *reinterpret_cast<uint2 *>(o4) = make_uint2(Elem<T>::pack2(y.x, y.y), Elem<T>::pack2(y.z, y.w));
        }
    };
    // record `slot` of a CTA: 0 its first item, 1 its last one; 2 and 3 the
    // merged record of the group of sharers that record 0 or 1 heads
    auto global_rec = [&](int c, int slot) { return p.records + ((int64_t)c * 4 + slot) * p.rec_floats; };

    // The CTA's records, in the items' order: lane r of every warp looks at
    // record r; a run of records of one item starts where the item changes.
    const int32_t mine = lane < 2 * W ? rec_first[lane] : -1;
    const uint32_t valid = __ballot_sync(0xffffffffu, mine >= 0);
    if (valid == 0) return;
    const uint32_t before = valid & ((1u << lane) - 1u);
    const int32_t prev = __shfl_sync(0xffffffffu, mine, before != 0 ? 31 - __clz(before) : lane);
    const bool starts_item = mine >= 0 && (before == 0 || prev != mine);
    const uint32_t starts = __ballot_sync(0xffffffffu, starts_item);
    const int groups = __popc(starts), first_group = __ffs(starts) - 1, last_group = 31 - __clz(starts);
    // whether the first and the last of the items lie partly with the CTAs before and behind
    const int32_t first_tile = rec_first[first_group] + kFp4Item, last_tile = rec_first[last_group] + kFp4Item;
    const int shared_first = first_tile < c0 ? first_group : -1;
    const int shared_last = last_tile >= c0 && last_tile + rec_n[last_group] > c1 ? last_group : -1;
    if (warp == 0) {
        if (mine >= 0)
            rec_at[__popc(before)] = smem_u32(smem) + ((lane & 1) ? (lane >> 1) * C::kRingBytes
                                                                  : W * C::kRingBytes + (lane >> 1) * C::kRec * 4);
        if (starts_item) group_rec[__popc(starts & ((1u << lane) - 1u))] = lane | __popc(before) << 8;
        if (lane == 0) group_rec[groups] = __popc(valid) << 8;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < groups * elements; i += C::kThreads) {
        const int g = i / elements, r0 = group_rec[g] & 255;
        float *dst = r0 == shared_first ? global_rec(cta, 0) : r0 == shared_last ? global_rec(cta, 1) : nullptr;
        merge(group_rec[g] >> 8, group_rec[g + 1] >> 8, rec_b[r0], rec_it[r0], dst, i - g * elements);
    }
    if (shared_first < 0 && shared_last < 0) return;

    // ---- items shared between CTAs -------------------------------------------
    // Warp k counts this CTA as one of the sharers of item k (0: shared with CTAs
    // before, 1: with CTAs behind), and the last of them merges their records.
    // Many sharers do so in two levels: the last of a group of neighbours merges
    // the group's, the last of the groups the groups'.
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {
        __threadfence();                       // all of the CTA's stores come before its counts
        __syncthreads();
        if (warp < 2) {
            const int k = warp, r0 = k ? shared_last : shared_first;
            int last = 0;
            if (r0 >= 0 && (level == 0 || arrived[k] == 2)) {
                const int32_t first = rec_first[r0] + kFp4Item;   // its first tile
                const int o0 = runs.owner(first), n = runs.owner(first + rec_n[r0] - 1) - o0 + 1;
                const bool two = n > C::kFlat, grouped = two && level == 0;
                const int g0 = grouped ? (cta - o0) / kFp4Group * kFp4Group : 0, gslot = g0 == 0 ? 1 : 0;
                const int sharers = grouped ? min(kFp4Group, n - g0) : two ? (n + kFp4Group - 1) / kFp4Group : n;
                int32_t *counter = grouped ? p.group_counters + (int64_t)(o0 + g0) * 2 + gslot
                                           : p.counters + (int64_t)rec_b[r0] * items_per_seq + rec_it[r0];
                if (lane == 0) {
                    last = atomicAdd(counter, 1) == sharers - 1;
                    if (last) *counter = 0;    // nobody else touches it again in this call
                    sharers_of[k] = sharers;
                    merged_to[k] = grouped ? global_rec(o0 + g0, 2 + gslot) : nullptr;
                }
                last = __shfl_sync(0xffffffffu, last, 0) * (grouped ? 2 : 1);
                // an item's record is its first CTA's last one and every other CTA's first one
                const int c = two && !grouped ? lane * kFp4Group : g0 + lane;
                if (lane < sharers) source[k][lane] = global_rec(o0 + c, (two && !grouped ? 2 : 0) + (c == 0 ? 1 : 0));
            }
            if (lane == 0) arrived[k] = last;  // 2: and there is another level
        }
        __syncthreads();
        const int a0 = arrived[0], a1 = arrived[1];
        if (a0 == 0 && a1 == 0) return;
        __threadfence();
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            if ((k ? a1 : a0) == 0) continue;
            // the records into shared memory, where the CTA's own have been merged, all of
            // them on their way at once
            constexpr int kPieces = C::kRec / 4;
            const int n = sharers_of[k], r0 = k ? shared_last : shared_first;
#pragma unroll 1
            for (int i = threadIdx.x; i < n * kPieces; i += C::kThreads) {
                const int r = i / kPieces;
                cp_async16(smem_u32(smem) + i * 16, source[k][r] + (i - r * kPieces) * 4);
            }
            if ((int)threadIdx.x < n) rec_at[threadIdx.x] = smem_u32(smem) + threadIdx.x * C::kRec * 4;
            cp_async_commit();
            cp_async_wait<0>();
            __syncthreads();
#pragma unroll 1
            for (int i = threadIdx.x; i < elements; i += C::kThreads)
                merge(0, n, rec_b[r0], rec_it[r0], merged_to[k], i);
            __syncthreads();                   // before the next records come
        }
        if (a0 < 2 && a1 < 2) return;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

template <typename T, int D, int NT, bool WHOLE>
struct Fp4Launch {
    using C = Fp4Cfg<T, D, NT>;
    static std::atomic<int> configured[64];

    static cudaError_t plan(int batch, int64_t max_tiles, Fp4Plan *plan) {
        auto kern = decode_fp4_kernel<T, D, NT, WHOLE>;
        const size_t smem = C::bytes(batch);
        cudaError_t e = ensure_smem_limit(kern, smem, configured);
        if (e != cudaSuccess) return e;
        int sms = 0;                               // what the limit allows, an SM holds
        e = device_sm_count(&sms);
        if (e != cudaSuccess) return e;
        const int64_t grid = sms < kFp4Groups * kFp4Group ? sms : kFp4Groups * kFp4Group;   // one CTA per SM
        const int64_t cap = (max_tiles + C::kWarps * kFp4MinTiles - 1) / (C::kWarps * kFp4MinTiles);
        const int64_t most = cap > plan->items ? cap : plan->items;   // an item to a CTA, or equal runs
        plan->grid = (int)(grid > most ? most : grid);
        plan->max_grid = (int)grid;
        plan->smem = smem;
        return cudaSuccess;
    }
    static cudaError_t launch(const Fp4Decode &p, const Fp4Plan &plan, cudaStream_t stream) {
        if (plan.grid <= 0) return cudaErrorInvalidValue;
        return launch_clustered(decode_fp4_kernel<T, D, NT, WHOLE>, plan.grid, C::kThreads, plan.smem, 1, stream, p,
                                plan.units_per_kv);
    }
};
template <typename T, int D, int NT, bool WHOLE> std::atomic<int> Fp4Launch<T, D, NT, WHOLE>::configured[64];

// f(Fp4Launch<...>{}) for the shape's instantiation.
template <typename T, typename F>
static cudaError_t dispatch_fp4_typed(int head_dim, int nt, bool whole, F &&f) {
    switch (head_dim) {
        case 64:
            if (whole) return nt == 2 ? f(Fp4Launch<T, 64, 2, true>{}) : f(Fp4Launch<T, 64, 1, true>{});
            return nt == 2 ? f(Fp4Launch<T, 64, 2, false>{}) : f(Fp4Launch<T, 64, 1, false>{});
        case 128:
            if (whole) return nt == 2 ? f(Fp4Launch<T, 128, 2, true>{}) : f(Fp4Launch<T, 128, 1, true>{});
            return nt == 2 ? f(Fp4Launch<T, 128, 2, false>{}) : f(Fp4Launch<T, 128, 1, false>{});
        case 256: return whole ? f(Fp4Launch<T, 256, 1, true>{}) : f(Fp4Launch<T, 256, 1, false>{});
    }
    return cudaErrorInvalidValue;
}
template <typename F>
static cudaError_t dispatch_fp4(int dtype, int head_dim, int nt, bool whole, F &&f) {
    switch (dtype) {
        case PA_F32: return dispatch_fp4_typed<float>(head_dim, nt, whole, f);
        case PA_F16: return dispatch_fp4_typed<__half>(head_dim, nt, whole, f);
        case PA_BF16: return dispatch_fp4_typed<__nv_bfloat16>(head_dim, nt, whole, f);
    }
    return cudaErrorInvalidValue;
}

cudaError_t plan_decode_fp4(int dtype, int head_dim, int group, int batch, int kv_heads, int block_size,
                            int64_t max_tiles_per_item, Fp4Plan *plan) {
    // one 8-column tile per item, or two when the kv head has more columns: the
    // conversion of a tile, not its MMAs, is what an item costs (32 x 2048 tokens,
    // 16 heads to each of 4: 20.1 us with two, 22.8 in two items of one)
    const int columns = group * (dtype == PA_F32 ? 2 : 1);
    plan->nt = head_dim <= 128 && columns > 8 ? 2 : 1;
    const int heads = plan->nt * 8 / (dtype == PA_F32 ? 2 : 1);
    plan->units_per_kv = (group + heads - 1) / heads;
    plan->items = (int64_t)batch * kv_heads * plan->units_per_kv;
    plan->whole_tiles = block_size % 16 == 0;
    const int64_t total = plan->items * max_tiles_per_item;
    if (total >= (int64_t)INT32_MAX / 2) return cudaErrorInvalidValue;
    return dispatch_fp4(dtype, head_dim, plan->nt, plan->whole_tiles, [&](auto l) { return l.plan(batch, total, plan); });
}

cudaError_t launch_decode_fp4(int dtype, const Fp4Decode &p, const Fp4Plan &plan, cudaStream_t stream) {
    return dispatch_fp4(dtype, p.d.D, plan.nt, plan.whole_tiles, [&](auto l) { return l.launch(p, plan, stream); });
}

}  // namespace pa
