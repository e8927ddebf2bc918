// chunk_umma.cu -- attention of several new tokens on the fifth-generation
// tensor cores (tcgen05.mma, scores, weights and outputs in tensor memory),
// 16-bit types, head_dim 64 and 128.
//
// An item is 256 query rows in two tiles of 128 (in the differential form 128
// rows, a tile for each map), a step a tile of 128 cache positions:
//     S_s = Q_s K^T                M = 128 rows, N = 128 positions, K = head_dim
//     O_s += P_s V                 M = 128 rows, N = head_dim, K = 128 positions
// with P_s = 2^(scale log2(e) (S_s - m)) by the 128 threads of tile s, a row
// each, between the two.  K and V arrive by TMA as 128-byte swizzled rows, K the
// K-major B operand of the first product, V the MN-major B operand of the
// second; P is the A operand of the second in tensor memory, over the columns that
// S had (at head_dim 64 there is room beside them for one part of the weights: 4
// prompts of 2048, 32 heads on 8, 121 us there, 123 here).  While the
// threads of one tile take the exponentials of a step the tensor core multiplies
// for the other.  An item of up to 128 rows (single tokens, ends of prompts) has
// its steps dealt to the two tiles in turn instead, and their states are joined
// at its end (of the item or of the CTA's share of it; 4 tokens behind 2048 in 32
// sequences, 64 heads, one part of weights: 66 us with two states to a share's record,
// 62 with one).
//
// What bounds it: long contexts, the tensor core (4096 tokens behind 28672, 64
// heads on 8 of 128: 2.75 ms back to back, 1.50 PFLOP/s of what is seen, 78% of a library
// product's rate in a burst); prompts, a step's way through both products and the
// exponentials, columns of the diagonal that are not seen, starts and ends of items (8 of
// 900 to 2047 tokens: 422 us, 1.07 PFLOP/s, the tensor core busy 56% of the time); few
// rows, the copies of K and V and 20 us of start, records and merge (32 x 4 tokens behind
// 2048: 67 us, 3.4 TB/s from memory); blocks that are copied row by row, the copying warp.
//
// Roles (512 threads): warps 0-3 and 4-7 the weights of tile 0 and 1; warp 8 the
// schedule and the copies of K and V; warps 9 and 10 the products of tile 0 and 1,
// warp 9 tensor memory; warp 11 the query rows; warps 12-15 the outputs, while the
// others are at the next item, and before that a look at those V tiles that not all
// rows see alike: positions that no row sees become zeros, and where another is
// not finite the rows' threads weigh that tile's values one by one, each only
// those it sees (the product would let 0 times them reach every row).
//
// The weights are rounded to the type on their way into the second product, at
// most half a step of themselves off, and summed as rounded: rows are normalised by
// what they were weighed with, so that a rounding that many weights share does not
// stay in the output (unrounded sums: 8 prompts of 900 to 2047 tokens 417 us, 422 so;
// 16 of 450 to 1000 with a window of 512 201 and 207).  An output that sums many of
// them is then as far from exact as its own rounding (1.4 times the error of an exact
// product's rounded result).  TWO: rounded weight and rest (in the columns that S has
// and P not), 1.0 times: in the differential form, where two such sums may all but
// cancel, and for few rows, so that they come out as from the decode (32 x 4 tokens behind
// 2048, 64 heads, 62 us with one part, 67 so).  Two parts for all would take the
// prompts to 530 us and 4096 tokens behind 28672 from 2.7 ms to 3.6.
//
// m is the maximum at the time it was last taken: O is rescaled only when a row's
// maximum has grown by more than 2^8 since, so weights stay below 2^8 and the sum
// of a row above 1.
#include <type_traits>

#include "chunk_sched.cuh"
#include "umma.cuh"

namespace pa {

namespace {

using namespace chunk;

constexpr int kThreads = 512;
constexpr int kKT = 128;                   // cache positions per tile
constexpr int kProducerWarp = 8, kMmaWarp = 9, kQWarp = 11, kOutWarp = 12;
constexpr float kLazy = 8.f;
constexpr int kItems = 4;                  // items of the schedule that roles may be apart

// What the roles know of an item: the CTA's share [k0, k1) of its steps, which
// steps each tile takes part in and what its rows see.
struct Share {
    int b, hk, n0, nrows;      // sequence, kv head, first row, rows
    int pos, lo;               // position of the sequence's first new token, first tile of positions
    int k0, k1;                // k0 < 0: no more items
    int cut;                   // the share is not the whole item
    int need_lo, need_hi;      // positions that some row sees
    int a[2], e[2];            // steps of each tile: a, a + stride, ... below e
    int stride;                // 2: both tiles are the same rows, with steps in turn
    int all_lo[2], all_hi[2];  // positions that all its rows see
    __device__ __forceinline__ int begin(int s) const { return s ? a[1] : a[0]; }
    __device__ __forceinline__ int finish(int s) const { return s ? e[1] : e[0]; }
    // not all rows see all positions of step k
    __device__ __forceinline__ bool partial(int k) const {
        const int t0 = (lo + k) * kKT;
        return t0 + kKT - 1 > all_hi[0] || t0 < all_lo[1];
    }
    template <bool DIFF>
    __device__ __forceinline__ void set(const ChunkParams &p, const Item &x, bool is_cut) {
        constexpr int R = DIFF ? 128 : 256;
        b = x.b;
        hk = x.hk;
        pos = x.pos;
        lo = x.lo;
        k0 = x.k0;
        k1 = x.k1;
        cut = is_cut;
        n0 = x.i * R;
        nrows = min(R, x.cnt * p.G - n0);
        need_lo = 0;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int r0 = DIFF ? 0 : s * 128, nr = min(128, nrows - r0);
            a[s] = e[s] = 0;
            if (s == 1) all_lo[1] = all_lo[0], all_hi[1] = all_hi[0];
            if (nr <= 0) continue;
            const int first = pos + (int)by_group(p, n0 + r0), last = pos + (int)by_group(p, n0 + r0 + nr - 1);
            const int seen = p.window > 0 ? max(0, first - p.window + 1) : 0;
            a[s] = max(k0, seen / kKT - lo);
            e[s] = max(a[s], min(k1, last / kKT + 1 - lo));
            all_hi[s] = first;
            all_lo[s] = p.window > 0 ? max(0, last - p.window + 1) : 0;
            if (s == 0) need_lo = seen;
            need_hi = last;
        }
        stride = !DIFF && nrows <= 128 ? 2 : 1;
        if (stride == 2) {
            a[1] = min(k0 + 1, k1);
            e[1] = k1;
        }
    }
};

// 32 columns of this thread's lane
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// Wait for this thread's loads.  The registers they fill pass through, so that
// nothing that uses them comes before the wait.
__device__ __forceinline__ void pin16(uint32_t *r) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
template <int N>
__device__ __forceinline__ void tmem_landed(uint32_t *r) {
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; i += 16) pin16(r + i);
}
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// D[tmem] (+)= A * B[smem] with A in shared or tensor memory.  Descriptors are
// given as their halves: only the low one, with the address, differs between the
// products of a tile.
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                        uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}"
        ::"r"(d_tmem), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                        bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
// As mbar_wait, in a loop of a few instructions: there are some thirty waits, and
// what the roles fetch besides their work they wait for (unrolled by 4, as the
// compiler will: 8 prompts of 900 to 2047 tokens, 64 heads: 454 us, 401 so).
__device__ __forceinline__ bool mbar_wait_loop(uint32_t bar, uint32_t parity) {
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitLimit; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return false;
}

// True in one lane of the warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
    return is != 0;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// a += the two 16-bit elements of w: an instruction each, where unpacking them first
// takes one more (8 prompts of 900 to 2047 tokens, 64 heads: 434 us, 422 so)
template <typename T>
__device__ __forceinline__ void add_halves(float2 &a, uint32_t w) {
    if constexpr (std::is_same<T, __half>::value)
        asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tadd.rn.f32.f16 %0, x, %0;\n\tadd.rn.f32.f16 %1, y, %1;\n\t}"
            : "+f"(a.x), "+f"(a.y) : "r"(w));
    else
        asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tadd.rn.f32.bf16 %0, x, %0;\n\tadd.rn.f32.bf16 %1, y, %1;\n\t}"
            : "+f"(a.x), "+f"(a.y) : "r"(w));
}

// Columns [0, N) of a row to memory: O_a f0, with BOTH + O_b f1, each times its
// element of w (null: 1); zeros if `zero`, nothing unless `there`.  32 bytes a store
// where rows are so aligned (wide): a row to a lane touches 32 lines with every
// store, and half as many stores take half the time.
template <typename T, int N, bool BOTH>
__device__ __forceinline__ void store_row(uint32_t o_a, uint32_t o_b, float f0, float f1, T *row, bool there, bool zero,
                                          const T *w, bool wide) {
#pragma unroll 1
    for (int c = 0; c < N; c += 16) {
        uint32_t a[16], b[16], x[8];
        tmem_ld16(o_a + c, a);
        if (BOTH) tmem_ld16(o_b + c, b);
        tmem_landed<16>(a);
        if (BOTH) pin16(b);
#pragma unroll
        for (int h = 0; h < 16; h += 8) {
            float wf[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) wf[i] = 1.f;
            if (BOTH && w != nullptr) Elem<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(w + c + h)), wf);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y0 = __uint_as_float(a[h + 2 * i]) * f0, y1 = __uint_as_float(a[h + 2 * i + 1]) * f0;
                if (BOTH) {
                    y0 = fmaf(__uint_as_float(b[h + 2 * i]), f1, y0) * wf[2 * i];
                    y1 = fmaf(__uint_as_float(b[h + 2 * i + 1]), f1, y1) * wf[2 * i + 1];
                }
                x[h / 2 + i] = zero ? 0u : Elem<T>::pack2(y0, y1);
            }
        }
        if (there) {
            if (wide) {
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + c), "r"(x[0]), "r"(x[1]),
                             "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                             : "memory");
            } else {
                *reinterpret_cast<uint4 *>(row + c) = make_uint4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<uint4 *>(row + c + 8) = make_uint4(x[4], x[5], x[6], x[7]);
            }
        }
    }
}

// A row's state to a record of 256 rows: O_a f0, with BOTH + O_b f1 (a factor of 0:
// nothing of it, whatever it holds), its maximum m and sum l.
template <int D, bool BOTH>
__device__ __forceinline__ void put_record(float *rec, int row, uint32_t o_a, uint32_t o_b, float f0, float f1, float m, float l,
                                           bool there) {
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
        uint32_t a[16], b[16];
        tmem_ld16(o_a + c, a);
        if (BOTH) tmem_ld16(o_b + c, b);
        tmem_landed<16>(a);
        if (BOTH) pin16(b);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = f0 == 0.f ? 0.f : __uint_as_float(a[j + i]) * f0;
                if (BOTH && f1 != 0.f) y[i] = fmaf(__uint_as_float(b[j + i]), f1, y[i]);
            }
            if (there) *reinterpret_cast<float4 *>(record_at(rec, 256, row, c + j)) = make_float4(y[0], y[1], y[2], y[3]);
        }
    }
    if (there) {
        rec[256 * D + row] = m;
        rec[256 * D + 256 + row] = l;
    }
}

// 128-byte swizzled rows: K and V tiles are [16 groups of 8 rows][D/64][8 rows]
// [128 bytes], query tiles [E/64 or 1][128 rows][128 bytes].
template <int D, bool DIFF>
struct Layout {
    static constexpr int E = DIFF ? D / 2 : D;
    static constexpr uint32_t kGroup = 8 * D * 2;             // 8 rows of K or V
    static constexpr uint32_t kTile = kKT * D * 2;
    static constexpr int kK = D == 128 ? 2 : 4, kV = D == 128 ? 3 : 4;   // tiles in flight or waiting
    // Words of a step are read until its second product is issued, and written anew from
    // the copy of K kBadRing steps on, which waits for the scores kK steps before itself;
    // those come after the second product of the step before them.
    static constexpr int kBadRing = D == 128 ? 4 : 8;
    static_assert(kBadRing >= kK + 2 && kBadRing > kV, "words of a step in use");
    static constexpr uint32_t kQSlab = 128 * 128;
    static constexpr int kQSlabs = E <= 64 ? 1 : E / 64;     // (rows of 64 elements stay whole in the differential form)
    static constexpr uint32_t kQTile = kQSlabs * kQSlab;
    static constexpr uint32_t kQ = 0;                         // two query tiles
    static constexpr uint32_t kKRing = 2 * kQTile, kVRing = kKRing + kK * kTile;
    static constexpr uint32_t kBars = kVRing + kV * kTile;
    enum {
        K_FULL = 0,                // [kK] the tile's copies have landed
        K_EMPTY = K_FULL + kK,     // [kK] the products that read it are done
        V_FULL = K_EMPTY + kK,     // [kV]
        V_EMPTY = V_FULL + kV,     // [kV]
        READY = V_EMPTY + kV,      // [kV] the tile has been looked over
        S_FULL = READY + kV,       // [2] scores
        P_HALF = S_FULL + 2,       // [2] weights of the first 64 positions
        P_FULL = P_HALF + 2,       // [2] all weights
        O_DONE = P_FULL + 2,       // [2] last product of an item
        O_FREE = O_DONE + 2,       // [2] its result has been read
        Q_FULL = O_FREE + 2,       // [2] query rows
        Q_FREE = Q_FULL + 2,       // [2]
        ITEM_FULL = Q_FREE + 2,    // [kItems] the item is there
        ITEM_EMPTY = ITEM_FULL + kItems,   // [kItems] all who need it are done with it
        ROWS_FULL = ITEM_EMPTY + kItems,   // [2] an item's sums and maxima of rows
        ROWS_FREE = ROWS_FULL + 2, // [2] have been read
        WARM = ROWS_FREE + 2,      // the weights' threads have been through a step
        TURN = WARM + 1,           // [2] the tensor core is tile s's to use
        END = TURN + 2,            // [2]
        NBARS = END + 2
    };
    static constexpr uint32_t kTmem = kBars + NBARS * 8;
    static constexpr uint32_t kBad = (kTmem + 4 + 15) & ~15u; // [kBadRing] a tile has bad table entries
    static constexpr uint32_t kBadRows = kBad + kBadRing * 4; // [kBadRing][4] then: a bit per row
    static constexpr uint32_t kOdd = kBadRows + kBadRing * 16;   // [kBadRing][4] a V tile's 32 rows are not all finite
    static constexpr uint32_t kItem = kOdd + kBadRing * 16;   // [kItems], and one of no rows
    static constexpr uint32_t kRows = (kItem + (kItems + 1) * sizeof(Share) + 15) & ~15u;   // [2][2][128] sums and maxima of rows
    static constexpr uint32_t kEnd = kRows + 2 * 2 * 128 * 4;
    static constexpr uint32_t kPre = kKRing;                  // before the first copy
    static constexpr size_t kBytes = kEnd;
    static constexpr uint32_t kColS = 0, kColO = 256;         // S_s at 128 s, O_s D columns each
    static constexpr uint32_t kRest = 64;                     // P_s over S_s: rounded weights, then what they leave
    static_assert(kBytes <= 232448, "shared memory per CTA");
    static_assert((kGroups + 1) * 8 <= kK * kTile, "the sums fit the ring");
};

}  // namespace

// ROWS: K and V are copied row by row (box_rows is 0), else in boxes.
// TWO: weights go into the second product in two parts, rounded weight and rest.
template <typename T, int D, bool DIFF, bool ROWS, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_umma_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ CUtensorMap qmap, const __grid_constant__ ChunkParams p, const int box_rows,
                      const int q_tokens) {
    using L = Layout<D, DIFF>;
    constexpr int E = L::E, R = DIFF ? 128 : 256;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t kIdescS = f16_idesc(kBf16, false, false, 128, kKT);
    constexpr uint32_t kIdescO = f16_idesc(kBf16, false, true, 128, D);
    using Schedule = Sched<R, kKT>;
    allow_dependents();
    extern __shared__ __align__(1024) unsigned char smem[];   // swizzled tiles: 1024-byte aligned
    const uint32_t sb = smem_u32(smem);
    auto bar = [&](int i) { return sb + L::kBars + i * 8; };
    volatile uint32_t *badm = reinterpret_cast<volatile uint32_t *>(smem + L::kBad);
    volatile uint32_t *badr = reinterpret_cast<volatile uint32_t *>(smem + L::kBadRows);
    volatile uint32_t *oddm = reinterpret_cast<volatile uint32_t *>(smem + L::kOdd);
    auto odd_words = [&](uint32_t step) {
        const volatile uint64_t *o = reinterpret_cast<const volatile uint64_t *>(oddm + step % L::kBadRing * 4);
        return o[0] | o[1];
    };
    int64_t *pre = reinterpret_cast<int64_t *>(smem + L::kPre);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::NBARS; ++i) {
            int count = 1;
            if (i >= L::READY && i < L::S_FULL) count = 4;            // the looking warps
            if (i >= L::K_EMPTY && i < L::K_EMPTY + L::kK) count = 2; // the products of both tiles
            if (i >= L::V_EMPTY && i < L::V_EMPTY + L::kV) count = 2;
            if (i == L::S_FULL || i == L::S_FULL + 1) count = 2;      // the products, and what their warp knows
            if (i == L::Q_FREE || i == L::Q_FREE + 1) count = 2;
            if (i >= L::P_HALF && i < L::O_DONE) count = 4;           // the warps of a tile
            if (i == L::O_FREE || i == L::O_FREE + 1) count = 4;      // the warps of the outputs
            if (i >= L::ROWS_FULL && i < L::WARM) count = 4;
            if (i == L::WARM) count = 8;
            if (i >= L::ITEM_EMPTY && i < L::ITEM_EMPTY + kItems) count = 15;   // 8 warps of weights, 2, 1, 4
            mbar_init(bar(i), count);
        }
        Share *none = reinterpret_cast<Share *>(smem + L::kItem) + kItems;
        *none = Share{};
        none->stride = none->k1 = none->e[0] = none->e[1] = 1;
        none->all_hi[0] = none->all_hi[1] = -1;    // as a tile that not all rows see alike
        if (!ROWS) {
            prefetch_tensormap(&kmap);
            prefetch_tensormap(&vmap);
        }
        if (q_tokens > 0) prefetch_tensormap(&qmap);
        mbar_init_fence();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(sb + L::kTmem, 512);
        tmem_relinquish();
        tc05_fence_before_sync();
    }
    __syncthreads();
    tc05_fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kTmem);
    const Share *ring = reinterpret_cast<const Share *>(smem + L::kItem);
    // A wait gave up.  Lanes may come to that apart: a warp votes before it does anything
    // together again.
    bool abort = false;
    // item i of the CTA, or null at the end (or after a wait that gave up)
    auto item = [&](uint32_t i) -> const Share * {
        if (!mbar_wait_loop(bar(L::ITEM_FULL + i % kItems), (i / kItems) & 1)) abort = true;
        abort = __any_sync(0xffffffffu, abort);
        const Share *x = ring + i % kItems;
        return abort || x->k0 < 0 ? nullptr : x;
    };
    auto item_done = [&](uint32_t i) { mbar_arrive(bar(L::ITEM_EMPTY + i % kItems)); };   // one lane of a warp

    if (warp >= kProducerWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        // what went before: tensor memory, barriers and the weights' first step wait for
        // none of it
        grid_dependency_wait();
        int per = 0, errors;
        if (p.B > kWarpSeqs)
            per = Schedule::build(p, pre, threadIdx.x - kProducerWarp * 32, kThreads - kProducerWarp * 32, 1, &errors);
        if (warp == kProducerWarp) {
            // lane s copies box s (box_rows positions) of each tile; table entries are
            // looked up a tile ahead
            Slices slices;
            Schedule it;
            bool has = p.B <= kWarpSeqs ? it.locate(p, slices, &errors) : it.locate(p, slices, pre, per);
            __syncwarp();
            fence_proxy_async_smem();              // the ring's copies come after the sums
            const int boxes = ROWS ? 0 : kKT / box_rows;
            const uint32_t box_bytes = (uint32_t)box_rows * D * 2;
            uint32_t g = 0, i = 0;
            auto put_cut = [&](bool any) {
                const int of_all = p.B <= kWarpSeqs ? all_errors(p, errors) : errors;
                if (lane == 0) p.cuts[blockIdx.x] = cut_entry<R, kKT>(p, it, any, slices, of_all);
            };
            auto publish = [&](bool stop) {
                if (i >= kItems && !mbar_wait_loop(bar(L::ITEM_EMPTY + i % kItems), (i / kItems - 1) & 1)) abort = true;
                abort = __any_sync(0xffffffffu, abort);
                Share *x = reinterpret_cast<Share *>(smem + L::kItem) + i % kItems;
                if (lane == 0) {
                    if (stop) x->k0 = -1;
                    else x->set<DIFF>(p, it.x, it.cut());
                    mbar_arrive(bar(L::ITEM_FULL + i % kItems));
                }
                __syncwarp();
                ++i;
                return x;
            };
            // Blocks that are not whole groups of 8 rows: rows of 16-byte copies by all
            // lanes.  A tile is given to the products when the next one has been begun.
            // Bound by this warp's copies (4 prompts of 1024 tokens, 32 heads on 8 of 128,
            // blocks of 3: 134 us, of 16, in boxes: 64; on mma.sync 243).
            uint32_t pending = 0;                  // barrier of the tile begun last
            auto landed = [&](uint32_t next) {
                if (pending != 0) {
                    if (next != 0) asm volatile("cp.async.wait_group 1;" ::: "memory");
                    else asm volatile("cp.async.wait_group 0;" ::: "memory");
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pending);
                }
                pending = next;
            };
            auto gather = [&](const Share &sh) {
                constexpr int C = D / 8, RPI = 32 / C;   // lanes of a row, rows at once
                const int need_lo = sh.need_lo, need_hi = sh.need_hi, ch = lane % C, first = lane / C;
                const uint32_t column = (uint32_t)((ch ^ first) & 7) << 4;   // of row `first` of 8; others' differ by their bits
                // blocks of rows lane + 32 j of tile k: -1 not needed, -2 bad
                auto look_up = [&](int k, int (&blk)[4]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = (it.x.lo + k) * kKT + lane + 32 * j;
                        blk[j] = -1;
                        if (k < it.x.k1 && t >= need_lo && t <= need_hi) {
                            blk[j] = __ldg(p.block_table + (int64_t)it.x.b * p.MB + (p.bs_shift >= 0 ? t >> p.bs_shift : t / p.bs));
                            if (blk[j] < 0 || blk[j] >= p.num_blocks) blk[j] = -2;
                        }
                    }
                };
                int ahead[4];
                look_up(it.x.k0, ahead);
                for (int k = it.x.k0; k < it.x.k1; ++k, ++g) {
                    int64_t at[4];                 // places
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = (it.x.lo + k) * kKT + lane + 32 * j;
                        const int in_block = p.bs_shift >= 0 ? t & (p.bs - 1) : t % p.bs;
                        at[j] = ahead[j];
                        if (at[j] >= 0) at[j] = at[j] * p.block_stride_bytes + ((int64_t)it.x.hk * p.bs + in_block) * (D * 2);
                    }
                    look_up(k + 1, ahead);
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t n = half ? L::kV : L::kK, slot = g % n, round = g / n;
                        if (round > 0 && !mbar_wait_loop(bar((half ? L::V_EMPTY : L::K_EMPTY) + slot), (round - 1) & 1)) abort = true;
                        abort = __any_sync(0xffffffffu, abort);
                        if (abort) return;
                        if (half == 0) {
                            uint32_t any = 0;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t rows = __ballot_sync(0xffffffffu, at[j] == -2);
                                if (lane == 0) badr[g % L::kBadRing * 4 + j] = rows;
                                any |= rows;
                            }
                            if (lane == 0) badm[g % L::kBadRing] = any;
                        }
                        const uint32_t dst = sb + (half ? L::kVRing : L::kKRing) + slot * L::kTile + (ch >> 3) * 1024 + first * 128;
                        const char *pool = (half ? p.v_pool : p.k_pool) + ch * 16;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t there = __ballot_sync(0xffffffffu, at[j] >= 0);
                            const int64_t from = at[j] < 0 ? 0 : at[j];
#pragma unroll 2
                            for (int q = 0; q < 4; ++q)    // groups of 8 rows
#pragma unroll
                                for (int u = 0; u < 8; u += RPI) {
                                    const int64_t o = __shfl_sync(0xffffffffu, from, q * 8 + u + first);
                                    cp16(dst + (j * 4 + q) * L::kGroup + u * 128 + (column ^ (u << 4)), pool + o,
                                         (there >> (q * 8 + u + first) & 1) != 0);
                                }
                        }
                        asm volatile("cp.async.commit_group;" ::: "memory");
                        landed(bar((half ? L::V_FULL : L::K_FULL) + slot));
                    }
                }
            };
            while (has && !abort) {
                const Share &sh = *publish(false);
                [[maybe_unused]] auto look_up = [&](int k, bool &needed) -> int32_t {   // row of the box, -1 bad
                    const int t = (it.x.lo + k) * kKT + lane * box_rows;
                    needed = k < it.x.k1 && lane < boxes && t <= sh.need_hi && t + box_rows > sh.need_lo;
                    if (!needed) return 0;
                    const int j = p.bs_shift >= 0 ? t >> p.bs_shift : t / p.bs;
                    const int32_t blk = __ldg(p.block_table + (int64_t)it.x.b * p.MB + j);
                    if (blk < 0 || (int64_t)blk >= p.num_blocks) return -1;
                    return blk * p.rows_per_block + it.x.hk * p.bs + (t - j * p.bs);
                };
                if constexpr (ROWS) {
                    gather(sh);
                } else {
                    bool needed, ahead_needed;
                    int32_t y = look_up(it.x.k0, needed);
                    for (int k = it.x.k0; k < it.x.k1 && !abort; ++k, ++g) {
                        const int32_t ahead = look_up(k + 1, ahead_needed);
                        const bool bad = needed && y < 0, take = needed && y >= 0;
                        const uint32_t bits = __ballot_sync(0xffffffffu, bad);
                        const uint32_t bytes = __reduce_add_sync(0xffffffffu, take ? box_bytes : 0u);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t n = half ? L::kV : L::kK, slot = g % n, round = g / n;
                            const uint32_t full = bar((half ? L::V_FULL : L::K_FULL) + slot);
                            if (round > 0 && !mbar_wait_loop(bar((half ? L::V_EMPTY : L::K_EMPTY) + slot), (round - 1) & 1)) abort = true;
                            abort = __any_sync(0xffffffffu, abort);
                            if (abort) break;
                            if (half == 0) {
                                if (bits != 0 && lane < 4) {           // a bit per row of a bad box
                                    uint32_t rows = 0;
#pragma unroll 1
                                    for (int j = 0; j < 32; j += 8) rows |= (bits >> (lane * 32 + j) / box_rows & 1) * (0xffu << j);
                                    badr[g % L::kBadRing * 4 + lane] = rows;
                                }
                                if (lane == 0) badm[g % L::kBadRing] = bits;
                                __syncwarp();
                            }
                            if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                            __syncwarp();
                            if (take) {
                                const uint32_t dst = sb + (half ? L::kVRing : L::kKRing) + slot * L::kTile + lane * box_bytes;
                                const CUtensorMap *map = half ? &vmap : &kmap;
                                if (D == 128) tma_4d_g2s(dst, map, 0, 0, 0, y >> 3, full);
                                else tma_2d_g2s(dst, map, 0, y, full);
                            }
                        }
                        y = ahead;
                        needed = ahead_needed;
                    }
                }
                if (i == 1) put_cut(true);
                has = it.next(p);
            }
            if (i == 0) put_cut(false);
            if (ROWS) landed(0);
            publish(true);
            // every copy has landed before the CTA may exit
            for (uint32_t u = g > L::kK ? g - L::kK : 0; u < g; ++u) mbar_wait_loop(bar(L::K_FULL + u % L::kK), (u / L::kK) & 1);
            for (uint32_t u = g > L::kV ? g - L::kV : 0; u < g; ++u) mbar_wait_loop(bar(L::V_FULL + u % L::kV), (u / L::kV) & 1);
        } else if (warp < kQWarp) {
            // Products of tile s.  The whole warp walks the steps, so that what the
            // products are given is known to be the same in all lanes; one lane issues
            // them.  The two warps take turns at the tensor core: while one issues, the
            // other walks on and waits, and the tiles stay half a step apart (left to
            // themselves both products, then both exponentials, run side by side).
            const int s = __shfl_sync(0xffffffffu, warp == kMmaWarp ? 0 : 1, 0);
            const bool leader = elect_one();
            // descriptors: 128-byte swizzling, version 1, distance of 8-row groups in the high half
            constexpr uint32_t kFlags = (1u << 14) | (2u << 29);
            constexpr uint32_t kQHi = kFlags | (1024 >> 4), kKvHi = kFlags | (L::kGroup >> 4);
            const uint32_t base = __shfl_sync(0xffffffffu, sb, 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t col_s = tm + L::kColS + s * 128, col_o = tm + L::kColO + s * D;
            const uint32_t q_lo = ((base + L::kQ) >> 4) + (DIFF && E < 64 ? s * (E * 2 >> 4) : 0);
            // of the slot
            uint32_t k_lo = ((base + L::kKRing) >> 4) + (DIFF ? (s * E >> 6) * (1024 >> 4) + ((s * E & 63) * 2 >> 4) : 0);
            uint32_t v_lo = ((base + L::kVRing) >> 4) | ((1024 >> 4) << 16);
            const uint32_t bars = base + L::kBars, of_s = s * 8;
            uint32_t step = 0, i = 0, ks = 0, vs = 0, items = 0, turns = 0;
            // a bit per barrier: the parity of the round that is waited for next
            uint32_t phase = 0;
            constexpr uint32_t kPhK = 1, kPhV = 2, kPhQ = 4, kPhP = 8, kPhO = 16, kPhT = 32, kPhQ1 = 64;
            if (!mbar_wait_loop(bar(L::WARM), 0)) abort = true;
            // A lane that gave up leaves the item's steps by itself; it meets the others at the
            // next item()'s vote (a vote at each step: 8 prompts of 900 to 2047 tokens 430 us,
            // 417 so).
            auto wait = [&](uint32_t b, uint32_t bit) {
                if (!mbar_wait_loop(b, (phase & bit) != 0)) abort = true;
                phase ^= bit;
            };
            for (const Share *x; (x = item(i)) != nullptr; ++i) {
                auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
                const int k0 = same(x->k0), k1 = same(x->k1), stride = same(x->stride);
                const int a = same(x->begin(s)), e = same(x->finish(s));
                const int qs = stride == 2 ? 0 : s;
                const bool q_shared = stride == 2 && k1 - k0 > 1;   // by both warps
                const bool q0_loaded = same(x->a[0] < x->e[0]) != 0;
                const uint32_t a_lo = q_lo + qs * (L::kQTile >> 4);
                if (leader) item_done(i);
                bool q_here = false;
                for (int k = k0 - stride; k < k1; ++k) {
                    const int kq = k + stride;
                    const bool pv = k >= k0, qk = kq < k1;
                    const bool turn = stride == 1 || ((k - k0) & 1) == s;
                    const bool w = pv && turn && k >= a && k < e, q = qk && turn && kq >= a && kq < e;
                    uint64_t odd = 0;
                    // what the batch needs, before its turn
                    if (pv) {
                        wait(bars + (L::READY + vs) * 8, kPhV);
                        if (vs != L::kV - 1) phase ^= kPhV;        // one parity for the ring's round
                    }
                    if (qk) {
                        wait(bars + (L::K_FULL + ks) * 8, kPhK);
                        if (ks != L::kK - 1) phase ^= kPhK;
                    }
                    if (q && !q_here) {
                        // (in turn on one query tile, both warps wait for each of its rounds)
                        wait(bars + (L::Q_FULL + qs) * 8, qs == s ? kPhQ : kPhQ1);
                        q_here = true;
                    }
                    if (w) {
                        odd = odd_words(step);
                        if (k == a && items++ > 0) wait(bars + L::O_FREE * 8 + of_s, kPhO);
                    }
                    if (w && !mbar_wait_loop(bars + L::P_HALF * 8 + of_s, (phase & kPhP) != 0)) abort = true;
                    if (turns > 0 || s == 1) wait(bars + L::TURN * 8 + of_s, kPhT);
                    ++turns;
                    tc05_fence_after_sync();
                    // S = Q K^T of step kq
                    auto score = [&]() {
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < E / 16; ++kk)
                                umma_ss(col_s, a_lo + (kk >> 2) * (L::kQSlab >> 4) + (kk & 3) * 2, kQHi,
                                        k_lo + (kk >> 2) * (1024 >> 4) + (kk & 3) * 2, kKvHi, kIdescS, kk > 0);
                            umma_commit(bars + L::S_FULL * 8 + of_s);
                            mbar_arrive(bars + L::S_FULL * 8 + of_s);
                            if (kq + stride >= e) {        // a tile of the queries is free when both warps say so
                                umma_commit(bars + (L::Q_FREE + qs) * 8);
                                if (!q_shared) mbar_arrive(bars + (L::Q_FREE + qs) * 8);
                            }
                        }
                    };
                    // 64 of the positions of O += P V
                    auto weigh = [&](int kk0, bool first) {
#pragma unroll
                        for (int kk = kk0; kk < kk0 + 4; ++kk) {
                            const uint32_t v = v_lo + kk * (2 * L::kGroup >> 4);
                            umma_ts(col_o, col_s + kk * 8, v, kKvHi, kIdescO, kk > kk0 || !first);
                            if (TWO) umma_ts(col_o, col_s + L::kRest + kk * 8, v, kKvHi, kIdescO, true);
                        }
                    };
                    if (w) {
                        // O += P V of step k
                        if (leader && odd == 0) weigh(0, k == a);
                        wait(bars + L::P_FULL * 8 + of_s, kPhP);
                        tc05_fence_after_sync();
                        if (leader) {
                            if (odd == 0) weigh(4, false);
                            if (k + stride >= e) umma_commit(bars + L::O_DONE * 8 + of_s);
                        }
                    }
                    if (q) score();
                    if (leader) mbar_arrive(bars + L::TURN * 8 + (of_s ^ 8));
                    if (pv) {
                        if (leader) umma_commit(bars + (L::V_EMPTY + vs) * 8);
                        v_lo += L::kTile >> 4;
                        ++step;
                        if (++vs == L::kV) vs = 0, v_lo -= L::kV * (L::kTile >> 4);
                    }
                    if (qk) {
                        if (leader) umma_commit(bars + (L::K_EMPTY + ks) * 8);
                        k_lo += L::kTile >> 4;
                        if (++ks == L::kK) ks = 0, k_lo -= L::kK * (L::kTile >> 4);
                    }
                    if (abort) break;
                }
                // rounds of query tile 0 that warp 10 had nothing of pass all the same
                if (s == 1 && q0_loaded && !(stride == 2 && q_here)) phase ^= kPhQ1;
            }
            // every product has completed before tensor memory is freed
            if (leader) umma_commit(bars + (L::END + s) * 8);
            mbar_wait_loop(bars + (L::END + s) * 8, 0);
            __syncwarp();
        } else if (warp == kQWarp) {
            // query rows (the scores of rows that are not there go nowhere): one copy a
            // slab where a tile is whole tokens, else rows of 16-byte copies
            uint32_t items[2] = {0, 0}, i = 0;
            for (const Share *x; (x = item(i)) != nullptr; ++i) {
                const int x_n0 = x->n0, nrows = x->nrows, b = x->b, hk = x->hk;
                const bool active[2] = {x->a[0] < x->e[0], x->a[1] < x->e[1] && x->stride == 1};
                __syncwarp();
                if (lane == 0) item_done(i);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (!active[s]) continue;
                    if (items[s] > 0 && !mbar_wait_loop(bar(L::Q_FREE + s), (items[s] - 1) & 1)) abort = true;
                    abort = __any_sync(0xffffffffu, abort);
                    if (abort) break;
                    const int r0 = DIFF ? 0 : s * 128, n0 = x_n0 + r0, nr = min(128, nrows - r0);
                    const uint32_t qb = sb + L::kQ + s * L::kQTile, full = bar(L::Q_FULL + s);
                    if (q_tokens > 0) {
                        if (lane == 0) {
                            mbar_arrive_expect_tx(full, (uint32_t)(L::kQSlabs * q_tokens * p.G * 128));
#pragma unroll
                            for (int h = 0; h < L::kQSlabs; ++h)
                                tma_4d_g2s(qb + h * L::kQSlab, &qmap, 0, hk * p.G, b * p.T + (int)by_group(p, n0),
                                           DIFF && E == 64 ? s : h, full);
                        }
                        __syncwarp();
                    } else {
                        constexpr int EQ = E < 64 ? 64 : E;      // elements of a row in the tile
                        constexpr int C = EQ / 8, RPI = 32 / C;  // lanes of a row, rows at once
                        const int ch = lane % C;
                        const T *src = reinterpret_cast<const T *>(p.q) + (int64_t)b * p.T * p.q_stride +
                                       (int64_t)hk * p.G * D + (DIFF && E == 64 ? s * E : 0) + ch * 8;
                        int t = (int)by_group(p, n0 + lane / C), h = (n0 + lane / C) - t * p.G;
#pragma unroll 4
                        for (int r = lane / C; r < nr; r += RPI) {
                            cp16(qb + (ch >> 3) * L::kQSlab + r * 128 + (((ch & 7) ^ (r & 7)) << 4), src + t * p.q_stride + h * D,
                                 true);
                            for (h += RPI; h >= p.G; h -= p.G) ++t;
                        }
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(full);
                    }
                    ++items[s];
                }
                if (abort) break;
            }
            // copies have landed before the CTA may exit
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (items[s] > 0) mbar_wait_loop(bar(L::Q_FULL + s), (items[s] - 1) & 1);
        } else {
            // V tiles, a row of a tile to a thread, then the item's outputs, a row to a
            // thread: tensor memory of the warp's quarter
            const int r = (warp & 3) * 32 + lane;
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const float *rows = reinterpret_cast<const float *>(smem + L::kRows);
            uint32_t g = 0, i = 0, done = 0;      // done: a parity for each tile
            auto wait = [&](uint32_t b, uint32_t parity) {
                if (!abort && !mbar_wait_loop(b, parity)) abort = true;
                abort = __any_sync(0xffffffffu, abort);
                return !abort;
            };
            const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
            // look over the V tile of step k of an item, tile g of the CTA
            auto look = [&](const Share &sh, int k) {
                    const uint32_t slot = g % L::kV;
                    if (!wait(bar(L::V_FULL + slot), (g / L::kV) & 1)) return;
                    const uint32_t bad = badm[g % L::kBadRing];
                    bool odd = false;
                    if (bad != 0 || sh.partial(k)) {
                        const int t = (sh.lo + k) * kKT + r;
                        uint4 *row = reinterpret_cast<uint4 *>(smem + L::kVRing + slot * L::kTile + (r >> 3) * L::kGroup + (r & 7) * 128);
                        const bool unseen = t < sh.need_lo || t > sh.need_hi || (bad != 0 && (badr[g % L::kBadRing * 4 + (warp & 3)] >> lane & 1) != 0);
                        // an exponent of all ones carries into the sign's place
                        constexpr uint32_t kOne = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
                        uint32_t carry = 0;
#pragma unroll 1
                        for (int h = 0; h < D / 64; ++h) {
                            uint4 v[8];
#pragma unroll
                            for (int c = 0; c < 8; ++c) v[c] = row[h * 64 + ((c + r) & 7)];   // neighbouring rows: other banks
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                carry |= ((v[c].x & 0x7fff7fffu) + kOne) | ((v[c].y & 0x7fff7fffu) + kOne) |
                                         ((v[c].z & 0x7fff7fffu) + kOne) | ((v[c].w & 0x7fff7fffu) + kOne);
                                if (unseen) row[h * 64 + c] = make_uint4(0, 0, 0, 0);
                            }
                        }
                        odd = !unseen && (carry & 0x80008000u) != 0;
                        fence_proxy_async_smem();
                    }
                    // the word was last read for step g - L::kBadRing, whose tile has left the ring
                    odd = __any_sync(0xffffffffu, odd);
                    if (lane == 0) {
                        oddm[g % L::kBadRing * 4 + (warp & 3)] = odd;
                        mbar_arrive(bar(L::READY + slot));
                    }
                    ++g;
            };
            int ahead = 0;                         // of the item's tiles, looked over already
            for (const Share *x = item(i); x != nullptr; ++i) {
                const Share &sh = *x;
                for (int k = sh.k0 + ahead; k < sh.k1 && !abort; ++k) look(sh, k);
                if (abort) break;
                // The next item's first tile before the outputs, or it would wait for them (8
                // prompts of 900 to 2047 tokens, 64 heads: 486 us after them, 445 so; two
                // tiles: 460).  Its copy waits for no output.
                const Share *following = item(i + 1);
                ahead = 0;
                if (following != nullptr) look(*following, following->k0 + ahead++);
                if (abort) break;
                const bool active[2] = {sh.a[0] < sh.e[0], sh.a[1] < sh.e[1]};
                float l[2] = {0.f, 0.f}, m[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (!active[s]) continue;
                    if (!wait(bar(L::ROWS_FULL + s), done >> s & 1)) break;
                    l[s] = rows[s * 256 + r];
                    m[s] = rows[s * 256 + 128 + r];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::ROWS_FREE + s));
                }
                if (abort) break;
                const bool same = DIFF || sh.stride == 2;          // both tiles are the same rows
                auto place = [&](int row, int &head) {             // of a row's output
                    const int n = sh.n0 + row, tok = (int)by_group(p, n);
                    head = sh.hk * p.G + n - tok * p.G;
                    return reinterpret_cast<T *>(p.out) + (((int64_t)sh.b * p.T + tok) * p.H + head) * D;
                };
                auto o_done = [&](int s) {
                    const bool ok = wait(bar(L::O_DONE + s), done >> s & 1);
                    done ^= 1u << s;
                    tc05_fence_after_sync();
                    return ok;
                };
                auto o_free = [&](int s) {
                    tc05_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::O_FREE + s));
                };
                const uint32_t o0 = tmem + lanes + L::kColO, o1 = o0 + D;
                auto rec = [&]() { return p.records + ((int64_t)blockIdx.x * 2 + (sh.k0 == 0)) * p.rec_floats; };
                if (!same || (DIFF && sh.cut)) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int row = same ? r : s * 128 + r;
                        const bool there = row < sh.nrows, has_o = s ? active[1] : active[0];
                        const float ls = s ? l[1] : l[0], ms = s ? m[1] : m[0];
                        if (has_o && !o_done(s)) break;
                        if (ls < 0.f && there) report(p.err_word, PA_DEVERR_BAD_BLOCK);
                        if (sh.cut) {
                            if (__any_sync(0xffffffffu, there))
                                put_record<D, false>(rec(), s * 128 + r, o0 + s * D, 0, has_o ? 1.f : 0.f, 0.f, ms, ls, there);
                        } else {
                            int head;
                            T *dst = place(row, head);
                            store_row<T, D, false>(o0 + s * D, 0, ls == 0.f ? 0.f : 1.f / ls, 0.f, dst, there, ls < 0.f, nullptr, wide);
                        }
                        if (has_o) o_free(s);
                    }
                    if (abort) break;
                } else {
                    const bool there = r < sh.nrows, zero = l[0] < 0.f || l[1] < 0.f;
                    if (!o_done(0) || (active[1] && !o_done(1))) break;
                    if (zero && there) report(p.err_word, PA_DEVERR_BAD_BLOCK);
                    if (__any_sync(0xffffffffu, there)) {
                        float f0, f1;
                        const T *w = nullptr;
                        if constexpr (DIFF) {
                            int head;
                            place(r, head);
                            f0 = l[0] == 0.f ? 0.f : p.out_scale / l[0];
                            f1 = there && l[1] != 0.f ? -__ldg(p.lambdas + head) * p.out_scale / l[1] : 0.f;
                            w = reinterpret_cast<const T *>(p.norm_weight);
                            if (w != nullptr) {
                                // (out_scale is in both: the squares are taken without it)
                                const float g0 = l[0] == 0.f ? 0.f : 1.f / l[0];
                                const float g1 = there && l[1] != 0.f ? -__ldg(p.lambdas + head) / l[1] : 0.f;
                                float sq = 0.f;
#pragma unroll 1
                                for (int c = 0; c < D; c += 16) {
                                    uint32_t a[16], b[16];
                                    tmem_ld16(o0 + c, a);
                                    tmem_ld16(o1 + c, b);
                                    tmem_landed<16>(a);
                                    pin16(b);
#pragma unroll
                                    for (int j = 0; j < 16; ++j) {
                                        const float y = fmaf(__uint_as_float(b[j]), g1, __uint_as_float(a[j]) * g0);
                                        sq = fmaf(y, y, sq);
                                    }
                                }
                                const float rs = 1.f / sqrtf(sq * (1.f / D) + p.eps);
                                f0 *= rs;
                                f1 *= rs;
                            }
                        } else {
                            const float M = fmaxf(m[0], m[1]);
                            f0 = merge_weight(m[0], M);
                            f1 = merge_weight(m[1], M);
                            const float sum = f0 * l[0] + f1 * l[1];
                            if (sh.cut) {          // one state of both tiles
                                put_record<D, true>(rec(), r, o0, o1, f0, active[1] ? f1 : 0.f, M, zero ? -1.f : sum, there);
                            } else {
                                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                                f0 *= inv;
                                f1 *= inv;
                            }
                        }
                        if (DIFF || !sh.cut) {
                            int head;
                            T *dst = place(r, head);
                            if (DIFF || active[1]) store_row<T, D, true>(o0, o1, f0, f1, dst, there, zero, w, wide);
                            else store_row<T, D, false>(o0, 0, f0, 0.f, dst, there, zero, nullptr, wide);
                        }
                    }
                    o_free(0);
                    if (active[1]) o_free(1);
                }
                __syncwarp();
                if (lane == 0) item_done(i);
                x = following;
            }
        }
    } else {
        // ------------------------------------------------------------------
        // the rows of tile s: thread r has row r, the tensor-memory lane of its
        // warp's quarter
        // ------------------------------------------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int s = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t col_s = tmem + lanes + L::kColS + s * 128, col_o = tmem + lanes + L::kColO + s * D;
        const float scale = p.scale_log2;
        uint32_t g = 0, i = 0, ns = 0, items = 0;
        float *rows = reinterpret_cast<float *>(smem + L::kRows);
        auto wait = [&](uint32_t b, uint32_t parity) {
            if (!abort && !mbar_wait_loop(b, parity)) abort = true;
            abort = __any_sync(0xffffffffu, abort);
            return !abort;
        };
        // The first time through is a step of no rows on whatever tensor memory holds,
        // while the first tiles are on their way: it fetches the instructions.
        bool warm = false;
        for (;;) {
            if (warm && !wait(bar(L::ITEM_FULL + i % kItems), (i / kItems) & 1)) break;
            const Share &sh = ring[warm ? i % kItems : kItems];
            if (sh.k0 < 0) break;
            const int stride = sh.stride;
            const int r0 = DIFF || stride == 2 ? 0 : s * 128, row = r0 + r, n = sh.n0 + row;   // row of the item
            const bool there = row < sh.nrows;
            const bool idle = warm && r0 + (warp & 3) * 32 >= sh.nrows;   // none of the warp's rows is
            const int pos = sh.pos + (int)by_group(p, n);
            const int row_hi = there ? pos : INT32_MAX;                // rows that are not there may see anything
            const int row_lo = there && p.window > 0 ? max(0, pos - p.window + 1) : 0;
            const int k_end = sh.finish(s), k_base = sh.k0, t_base = sh.lo * kKT;
            const int all_hi = sh.all_hi[s], all_lo = sh.all_lo[s], item_hi = sh.all_hi[0], item_lo = sh.all_lo[1];
            float m = -INFINITY, l = 0.f;
            bool row_bad = false;
            for (int k = sh.begin(s); k < k_end; k += stride) {
                if (warm) {
                    if (!wait(bar(L::S_FULL + s), ns & 1)) break;
                    ++ns;
                }
                if (idle) {
                    if (lane == 0) {
                        mbar_arrive(bar(L::P_HALF + s));
                        mbar_arrive(bar(L::P_FULL + s));
                    }
                    continue;
                }
                tc05_fence_after_sync();
                uint32_t v[128];
                auto f = [&v](int i) { return __uint_as_float(v[i]); };
                const uint32_t step = g + (uint32_t)(k - k_base);
                const uint32_t bad = badm[step % L::kBadRing];
                const int t0 = t_base + k * kKT;
                // Code that runs seldom is kept in loops: what it costs is its fetch (the
                // first step of a launch takes four times the others).
                if (t0 + kKT - 1 > all_hi || t0 < all_lo) {
                    const int lo = row_lo - t0;
                    const uint32_t range = (uint32_t)(row_hi - row_lo);
#pragma unroll 1
                    for (int c = 0; c < kKT; c += 32) {
                        uint32_t x[32];
                        tmem_ld32(col_s + c, x);
                        tmem_landed<32>(x);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if ((uint32_t)(c + i - lo) > range) x[i] = 0xff800000u;
                        tmem_st16(col_s + c, x);
                        tmem_st16(col_s + c + 16, x + 16);
                    }
                    tmem_wait_st();
                }
                // the maximum of the first half while the second is on its way
                tmem_ld32(col_s, v);
                tmem_ld32(col_s + 32, v + 32);
                tmem_landed<64>(v);
                tmem_ld32(col_s + 64, v + 64);
                tmem_ld32(col_s + 96, v + 96);
                float m4[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) m4[j] = fmaxf(f(j), f(j + 4));
#pragma unroll
                for (int i = 8; i < 64; i += 8)
#pragma unroll
                    for (int j = 0; j < 4; ++j) m4[j] = fmaxf(m4[j], fmaxf(f(i + j), f(i + 4 + j)));
                tmem_landed<64>(v + 64);
                if (bad != 0) {
#pragma unroll 1
                    for (int c = 0; c < kKT; c += 32) {            // of 32 positions, those it sees
                        const int b0 = max(0, row_lo - t0 - c), b1 = min(31, row_hi - t0 - c);
                        if (b0 <= b1 && (badr[step % L::kBadRing * 4 + c / 32] >> b0 << b0 & (0xffffffffu >> (31 - b1))) != 0)
                            row_bad = true;
                    }
                }
#pragma unroll
                for (int i = 64; i < 128; i += 8)
#pragma unroll
                    for (int j = 0; j < 4; ++j) m4[j] = fmaxf(m4[j], fmaxf(f(i + j), f(i + 4 + j)));
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                // the last step's second product was issued before these scores: it is done
                const bool grown = (mx - m) * scale > kLazy;
                if (__any_sync(0xffffffffu, grown)) {
                    const float alpha = grown ? ex2_approx((m - mx) * scale) : 1.f;
                    if (grown) m = mx;
                    l *= alpha;
                    if (k > sh.begin(s)) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(col_o + c, o);
                            tmem_landed<16>(o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st16(col_o + c, o);
                        }
                    }
                }
                const float nb = m == -INFINITY ? 0.f : -m * scale;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    uint32_t w[16], rest[TWO ? 16 : 1];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 e = fma2(make_float2(f(c + 2 * i), f(c + 2 * i + 1)), make_float2(scale, scale), make_float2(nb, nb));
                        e.x = ex2_approx(e.x);
                        e.y = ex2_approx(e.y);
                        // the sum: of the weights that the product uses (two parts: but for the rest's rounding)
                        if (TWO) sum[i & 1] = add2(sum[i & 1], e);
                        w[i] = Elem<T>::pack2(e.x, e.y);
                        if (TWO) {
                            float2 r;
                            Elem<T>::unpack2(w[i], r.x, r.y);
                            rest[i] = Elem<T>::pack2(e.x - r.x, e.y - r.y);
                        } else {
                            add_halves<T>(sum[i & 1], w[i]);
                        }
                    }
                    tmem_st16(col_s + c / 2, w);
                    if (TWO) tmem_st16(col_s + L::kRest + c / 2, rest);
                    if (c == 32) {                 // the product of the first 64 positions may begin
                        tmem_wait_st();
                        tc05_fence_before_sync();
                        __syncwarp();
                        if (lane == 0 && warm) mbar_arrive(bar(L::P_HALF + s));
                    }
                }
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
                tmem_wait_st();
                if (warm && (bad != 0 || t0 + kKT - 1 > item_hi || t0 < item_lo)) {
                    const uint32_t slot = step % L::kV;
                    if (!wait(bar(L::READY + slot), (step / L::kV) & 1)) break;
                    if (odd_words(step) != 0) {
                        // O of the first step: once the last item's has been read
                        if (k == sh.begin(s) && items > 0) {
                            if (!wait(bar(L::O_FREE + s), (items - 1) & 1)) break;
                            tc05_fence_after_sync();
                        }
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t o32[32];
                            float o[32];
                            tmem_ld32(col_o + c0, o32);
                            tmem_landed<32>(o32);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = k > sh.begin(s) ? __uint_as_float(o32[i]) : 0.f;
#pragma unroll 1
                            for (int t = 0; t < kKT; ++t) {
                                uint32_t w2, rest = 0;
                                tmem_ld1(col_s + t / 2, w2);
                                if (TWO) tmem_ld1(col_s + L::kRest + t / 2, rest);
                                tmem_wait_ld();
                                asm volatile("" : "+r"(w2), "+r"(rest));
                                float w[2], r[2];
                                Elem<T>::unpack2(w2, w[0], w[1]);
                                Elem<T>::unpack2(rest, r[0], r[1]);
                                const float wt = (t & 1) ? w[1] + r[1] : w[0] + r[0];
                                const bool sees = t0 + t >= row_lo && t0 + t <= row_hi;
                                const unsigned char *vr = smem + L::kVRing + slot * L::kTile + (t >> 3) * L::kGroup +
                                                          (c0 >> 6) * 1024 + (t & 7) * 128;
#pragma unroll
                                for (int h = 0; h < 4; ++h) {
                                    const int ch = ((c0 & 63) >> 3) + h;
                                    const uint4 q = *reinterpret_cast<const uint4 *>(vr + ((ch ^ (t & 7)) << 4));
                                    float e[8];
                                    Elem<T>::unpack(q, e);
#pragma unroll
                                    for (int i = 0; i < 8; ++i) o[h * 8 + i] = sees ? fmaf(wt, e[i], o[h * 8 + i]) : o[h * 8 + i];
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 32; i += 16) {
                                uint32_t t[16];
#pragma unroll
                                for (int j = 0; j < 16; ++j) t[j] = __float_as_uint(o[i + j]);
                                tmem_st16(col_o + c0 + i, t);
                            }
                        }
                        tmem_wait_st();
                    }
                }
                tc05_fence_before_sync();
                __syncwarp();
                if (lane == 0 && warm) mbar_arrive(bar(L::P_FULL + s));
            }
            if (!warm) {
                if (lane == 0) mbar_arrive(bar(L::WARM));
                warm = true;
                continue;
            }
            g += (uint32_t)(sh.k1 - sh.k0);
            if (abort) break;
            if (sh.begin(s) < k_end) {             // sums and maxima to the warps of the outputs
                if (items > 0 && !wait(bar(L::ROWS_FREE + s), (items - 1) & 1)) break;
                ++items;
                rows[s * 256 + r] = row_bad ? -1.f : l;
                rows[s * 256 + 128 + r] = m == -INFINITY ? -INFINITY : m * scale;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::ROWS_FULL + s));
            }
            __syncwarp();
            if (lane == 0) item_done(i);
            ++i;
        }
    }
    if (abort && lane == 0) report(p.err_word, PA_DEVERR_TIMEOUT);
    __syncwarp();
    tc05_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc05_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

namespace {

template <typename T, int D, bool DIFF, bool ROWS, bool TWO>
cudaError_t plan_one(ChunkPlan *plan) {
    static std::atomic<int> limit[64];
    int sms = 0;
    cudaError_t e = ensure_smem_limit(chunk_umma_kernel<T, D, DIFF, ROWS, TWO>, Layout<D, DIFF>::kBytes, limit);
    if (e != cudaSuccess) return e;
    e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    plan->grid = sms;
    plan->maps = DIFF ? 2 : 1;
    plan->rows = 256 / plan->maps;
    plan->two_parts = TWO;
    plan->rec_floats = chunk_rec_floats(256, D);
    return cudaSuccess;
}

template <typename T, int D, bool DIFF, bool ROWS, bool TWO>
cudaError_t launch_one(const ChunkParams &p, const ChunkPlan &plan, cudaStream_t stream, const CUtensorMap &kmap,
                       const CUtensorMap &vmap, int box_rows, const CUtensorMap &qmap, int q_tokens) {
    return launch_clustered(chunk_umma_kernel<T, D, DIFF, ROWS, TWO>, plan.grid, kThreads, Layout<D, DIFF>::kBytes, 1, stream, kmap,
                            vmap, qmap, p, box_rows, q_tokens);
}

template <typename T, int D, typename F>
cudaError_t with_form(bool diff, bool rows, bool two, F f) {
    if (diff) return rows ? f.template operator()<T, D, true, true, true>() : f.template operator()<T, D, true, false, true>();
    if (two) return rows ? cudaErrorInvalidValue : f.template operator()<T, D, false, false, true>();
    return rows ? f.template operator()<T, D, false, true, false>() : f.template operator()<T, D, false, false, false>();
}
template <typename F>
cudaError_t with_kernel(int dtype, int head_dim, bool diff, bool rows, bool two, F f) {
    if (dtype == PA_F16)
        return head_dim == 64 ? with_form<__half, 64>(diff, rows, two, f) : with_form<__half, 128>(diff, rows, two, f);
    return head_dim == 64 ? with_form<__nv_bfloat16, 64>(diff, rows, two, f)
                          : with_form<__nv_bfloat16, 128>(diff, rows, two, f);
}

struct Planner {
    ChunkPlan *plan;
    template <typename T, int D, bool DIFF, bool ROWS, bool TWO>
    cudaError_t operator()() const { return plan_one<T, D, DIFF, ROWS, TWO>(plan); }
};
struct Launcher {
    const ChunkParams &p;
    const CUtensorMap &kmap, &vmap, &qmap;
    int box_rows, q_tokens;
    const ChunkPlan &plan;
    cudaStream_t stream;
    template <typename T, int D, bool DIFF, bool ROWS, bool TWO>
    cudaError_t operator()() const { return launch_one<T, D, DIFF, ROWS, TWO>(p, plan, stream, kmap, vmap, box_rows, qmap, q_tokens); }
};

}  // namespace

bool chunk_umma_supported(int dtype, int head_dim) {
    return (dtype == PA_F16 || dtype == PA_BF16) && (head_dim == 64 || head_dim == 128);
}

cudaError_t plan_chunk_umma(int dtype, int head_dim, bool diff, bool two_parts, int box_rows, ChunkPlan *plan) {
    return with_kernel(dtype, head_dim, diff, box_rows == 0, two_parts, Planner{plan});
}

cudaError_t launch_chunk_umma(int dtype, int head_dim, const ChunkParams &p, const CUtensorMap &kmap, const CUtensorMap &vmap,
                              int box_rows, const CUtensorMap &qmap, int q_tokens, const ChunkPlan &plan,
                              cudaStream_t stream) {
    return with_kernel(dtype, head_dim, plan.maps == 2, box_rows == 0, plan.two_parts,
                       Launcher{p, kmap, vmap, qmap, box_rows, q_tokens, plan, stream});
}

}  // namespace pa
