// Building blocks of the grouped products' kernels (mm.hip, mm_stream.hip, mm_mid.hip,
// mm_thin.hip).
//
//   kind 0  y[r, n]     = sum_k x[r, k] w[e, k, n]     (rows r of group e)
//   kind 1  dx[r, k]    = sum_n dy[r, n] w[e, k, n]
//   kind 2  dw[e, k, n] = sum_r x[r, k] dy[r, n]       (r over the rows of group e)
//   kind 3  y[r, n]     = (sum_k xq[r, k] wq[e, n, k]) xs[r] ws[e, n]     (int8)
//
// and two variants for the experts' gated projections:
//
//   kind 0, gated    h[r, f]  = SiLU(sum_k x[r, k] w_in[e, k, f]) sum_k x[r, k] w_up[e, k, f]: a tile's B
//                    operand is half as many columns of each matrix, side by side in LDS, and
//                    a wavefront holds the same columns of both products
//   kind 1, two      dx[r, k] = sum_f da[r, f] w_in[e, k, f] + db[r, f] w_up[e, k, f]: one contraction, whose
//                    steps run through the first pair of operands, then through the second
//
// The first reads x once for both projections and writes neither where no gradient is to follow;
// the second adds in fp32 what two products would round and add again.  64 experts, 16384 rows,
// 2048 x 1408, bf16: h 209 us (two products and the activation 293), dx 190 (two products and their
// sum 254); 8192^3 1607 us, 1370 TFLOP/s (1578), and dx 1626 (1695).
//
// All are C[i, j] = sum_c A[i, c] B[c, j] on tiles of C, in steps of the contraction that
// take 64 bytes of each index (32 bf16, 64 int8, 16 fp32).  An operand lies in memory in
// one of two layouts:
//   rows      the contraction runs along memory (x and dy of kinds 0, 1, 3; w of kind 1; wq).
//             In LDS a tile index keeps its 64 bytes as four 16-byte chunks, chunk q of index
//             m at q ^ swa4(m); a matrix operand is one ds_read_b128.
//   columns   the tile index runs along memory (w of kind 0; both operands of kind 2).  In LDS
//             a contraction index keeps its tile's values in a row, as in memory, bf16 with
//             32-byte blocks swizzled by the row; a matrix operand is two ds_read_b64_tr_b16
//             (bf16: each turns 4 rows x 16 columns) or four ds_read_b32 (fp32).
// In registers a matrix operand of 16 indexes is 16 bytes per lane: lane l holds index l & 15
// and contraction chunk l >> 4.  bf16 and int8 take it in one instruction (16x16x32,
// 16x16x64), fp32 in four (16x16x4; instruction i sums the contraction indexes 4 q + i, in
// both operands alike).
//
// Operands travel from memory straight into LDS (buffer loads of 16 bytes a lane, 1 KB a
// wavefront).  Loads past the tile's indexes or the contraction's end carry an offset past
// the buffer's end and read zeros: nothing of a neighbouring row, column or group enters a
// sum, and no select is needed after the load.
#pragma once

#include <type_traits>

#include "act.h"
#include "common.h"
#include "launch.h"
#include "mm_common.h"
#include "mm_launch.h"

namespace moe {

typedef short v4i16_t __attribute__((ext_vector_type(4)));
typedef short v8i16_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

enum class Elem { bf16, i8, f32 };

enum class Var { plain, gated, two };

template <int KIND_, Elem E_, Var V_ = Var::plain>
struct Op {
    static constexpr bool kGated = V_ == Var::gated, kTwo = V_ == Var::two;
    static_assert(!(kGated && KIND_ != 0) && !(kTwo && KIND_ != 1), "the variants of kinds 0 and 1");
    static constexpr int KIND = KIND_;
    static constexpr Elem ELEM = E_;
    static constexpr bool kACols = KIND == 2, kBCols = KIND == 0 || KIND == 2;
    static constexpr int ES = E_ == Elem::bf16 ? 2 : E_ == Elem::i8 ? 1 : 4;       // bytes of an element
    static constexpr int kStep = 64 / ES;                                          // contraction indexes a step
    using Acc = std::conditional_t<E_ == Elem::i8, i32x4_t, f32x4_t>;
};

__device__ __forceinline__ void lds_barrier() { asm volatile("s_barrier" ::: "memory"); }
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }      // lgkmcnt(0)
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uni(uint64_t v) {
    return ((uint64_t)(uint32_t)uni((int)(v >> 32)) << 32) | (uint32_t)uni((int)(uint32_t)v);
}

// Block swizzle of row k of a bf16 `columns` step with rows of RB bytes: the 32-byte block b
// sits at b ^ blk_swz(k).  One LDS cycle of a ds_read_b64_tr_b16 serves one block of the rows
// k0..k0+3 and k0+8..k0+11; the swizzle puts those eight on distinct banks (256 bytes a
// cycle; rows of 32 bytes leave no room for it).
template <int RB>
__device__ __forceinline__ int blk_swz(int k) {
    if constexpr (RB >= 256) return (k & 3) | (((k >> 3) & 1) << 2);
    else if constexpr (RB == 128) return ((k >> 1) & 1) | (((k >> 3) & 1) << 1);
    else if constexpr (RB == 64) return (k >> 3) & 1;
    else return 0;
}

// Swizzle of `rows` operands read 32 indexes at a time (mm_fp8.hip): the 16 lanes that one LDS
// cycle of a ds_read_b128 serves (see swa4) have four indexes each of every m mod 4, whose m / 4
// differ modulo 4.
__device__ __forceinline__ int swa32(int m) { return (m >> 2) & 3; }

// One operand of a tile of T indexes: what a wavefront needs to start the loads of a step.
// N loads of 1 KB each are this wavefront's (of the T / 16 that fill a step's stage).  R32: laid
// out for reads of 32 indexes.
template <int ES, bool COLS, int T, int N, bool R32 = false>
struct Operand {
    static constexpr int kRowB = T * ES;          // columns: bytes of a stage's row
    static constexpr int kStep = 64 / ES;
    uint64_t base;            // first byte of the tile: of its first index (rows) or of its first contraction row
    uint32_t ld;              // bytes from one memory row to the next
    uint32_t n;               // rows: indexes of the tile that exist; columns: contraction length
    uint32_t cbytes;          // rows: bytes of the contraction
    uint32_t off[N];          // this lane's offsets at step 0
    uint32_t kq;              // rows: this lane's byte within the step

    // first: this wavefront's first load; valid: indexes of the tile that exist
    __device__ __forceinline__ void plan(int first, int lane, int valid) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int j = first + i;
            if constexpr (COLS) {
                const int pos = j * 1024 + lane * 16;
                int k = pos / kRowB, c = (pos % kRowB) / 16;
                if constexpr (ES == 4 && T == 32) k ^= (k >> 3) & 1;
                if constexpr (ES == 2) c ^= 2 * blk_swz<kRowB>(k);
                else c ^= 4 * ((k >> 2) & (T == 32 ? 1 : 3));
                off[i] = c * (16 / ES) < valid ? (uint32_t)k * ld + (uint32_t)c * 16 : kOOB;
            } else {
                const int r = j * 16 + (lane >> 2), q = (lane & 3) ^ (R32 ? swa32(r) : swa4(r));
                kq = (uint32_t)q * 16;            // the same for every load: the swizzles' periods divide 16
                off[i] = r < valid ? (uint32_t)r * ld + kq : kOOB;
            }
        }
    }
    __device__ __forceinline__ void load(lds_char* stage, int first, int kt) const {
        if constexpr (COLS) {
            // (as scalar minima: a clamp or a saturating difference would be a vector instruction,
            // and the resource, then in vector registers, cost a loop over the lanes)
            uint32_t k0 = min((uint32_t)kt * kStep, n);
            asm("" : "+s"(k0));
            const uint32_t bytes = min(n - k0, (uint32_t)kStep) * ld;
            const __amdgpu_buffer_rsrc_t r = make_rsrc((const void*)(base + (uint64_t)kt * kStep * ld), bytes);
#pragma unroll
            for (int i = 0; i < N; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(stage + (first + i) * 1024), 16, off[i], 0, 0, 0);
        } else {
            // the step's place as the scalar offset: a lane's own is fixed, but for the end of the
            // contraction
            const uint32_t k0 = min((uint32_t)kt * 64, cbytes), left = cbytes - k0;
            const __amdgpu_buffer_rsrc_t r = make_rsrc((const void*)base, n * ld);
#pragma unroll
            for (int i = 0; i < N; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(stage + (first + i) * 1024), 16,
                                                         kq < left ? off[i] : kOOB, (int)k0, 0, 0);
        }
    }
};

// The B operand of a gated tile: T / 2 columns of one matrix, then of the other; N loads in all.
template <int ES, int T, int N>
struct GatedOperand {
    Operand<ES, true, T / 2, N / 2> in, up;
    __device__ __forceinline__ void plan(int first, int lane, int valid) {
        in.plan(first / 2, lane, valid);
        up.plan(first / 2, lane, valid);
    }
    __device__ __forceinline__ void load(lds_char* stage, int first, int kt) const {
        in.load(stage, first / 2, kt);
        up.load(stage + T / 2 * 64, first / 2, kt);
    }
};

// An operand whose steps run through one tensor and then, from step `half` on, through another
// of the same layout.
template <int ES, int T, int N>
struct TwoOperand {
    Operand<ES, false, T, N> o;
    uint64_t base2;
    int half;
    __device__ __forceinline__ void plan(int first, int lane, int valid) { o.plan(first, lane, valid); }
    __device__ __forceinline__ void load(lds_char* stage, int first, int kt) const {
        Operand<ES, false, T, N> p = o;
        if (kt >= half) p.base = base2;
        p.load(stage, first, kt >= half ? kt - half : kt);
    }
};

// 16-index block `blk` of an operand's stage as a matrix operand.
template <int ES, bool COLS, int T>
struct Reader {
    static constexpr int kRowB = T * ES;
    int rd, g, up = 0;
    __device__ __forceinline__ explicit Reader(int lane) {
        const int l16 = lane & 15, lq = lane >> 4;
        g = 0;
        if constexpr (COLS && ES == 2) {
            g = blk_swz<kRowB>(8 * lq + (l16 >> 2));          // the same for the rows of the second read, 4 further
            rd = (8 * lq + (l16 >> 2)) * kRowB + ((l16 & 3) << 3);
        } else if constexpr (COLS) {
            // One read takes a 64-byte block of four rows 4 apart, on four places of 256 bytes:
            // blocks trade places in fours, or where a row has two (T = 32), in twos, and the
            // rows of the upper half with their neighbours.
            static_assert(T % 64 == 0 || T == 32, "two blocks a row, or fours of them");
            g = T == 32 ? lq & 1 : lq;
            rd = 4 * lq * kRowB + l16 * 4;
            up = T == 32 ? (lq >> 1) * kRowB : 0;
        } else {
            rd = l16 * 64 + ((lq ^ swa4(l16)) << 4);
        }
    }
    __device__ __forceinline__ u32x4_t operator()(const lds_char* stage, int blk) const {
        if constexpr (COLS && ES == 2) {
            constexpr int M = kRowB >= 256 ? 7 : kRowB / 32 - 1;
            const lds_char* p = stage + rd + (((blk & ~M) | ((blk & M) ^ g)) << 5);
            const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16_t*)p);
            const v4i16_t hi =
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16_t*)(p + 4 * kRowB));
            const v8i16_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            return __builtin_bit_cast(u32x4_t, v);
        } else if constexpr (COLS) {
            typedef const __attribute__((address_space(3))) uint32_t lds_u32;
            const lds_char* at = stage + rd + ((blk & ~3) | ((blk & 3) ^ g)) * 64;
            if constexpr (T == 32) {
                lds_u32 *even = (lds_u32*)(at + up), *odd = (lds_u32*)(at - up);
                return u32x4_t{even[0], odd[kRowB / 4], even[2 * (kRowB / 4)], odd[3 * (kRowB / 4)]};
            }
            lds_u32* p = (lds_u32*)at;
            return u32x4_t{p[0], p[kRowB / 4], p[2 * (kRowB / 4)], p[3 * (kRowB / 4)]};
        } else {
            return *(const __attribute__((address_space(3))) u32x4_t*)(stage + rd + blk * 1024);
        }
    }
};

// Of a gated tile of T columns in all, FN blocks a wavefront: its block j < FN / 2 is of the first
// matrix, j >= FN / 2 of the second.
template <int ES, int T, int FN>
struct GatedReader {
    Reader<ES, true, T / 2> r;
    __device__ __forceinline__ explicit GatedReader(int lane) : r(lane) {}
    __device__ __forceinline__ u32x4_t operator()(const lds_char* stage, int blk) const {
        const int w = blk / FN, j = blk % FN;
        return r(stage + j / (FN / 2) * (T / 2 * 64), w * (FN / 2) + j % (FN / 2));
    }
};

template <typename O, int T, int N, bool R32 = false>
using OperandA = std::conditional_t<O::kTwo, TwoOperand<O::ES, T, N>, Operand<O::ES, O::kACols, T, N, R32>>;
template <typename O, int T, int N, bool R32 = false>
using OperandB = std::conditional_t<O::kTwo, TwoOperand<O::ES, T, N>,
                                    std::conditional_t<O::kGated, GatedOperand<O::ES, T, N>, Operand<O::ES, O::kBCols, T, N, R32>>>;
template <typename O, int T, int FN>
using ReaderB = std::conditional_t<O::kGated, GatedReader<O::ES, T, FN>, Reader<O::ES, O::kBCols, T>>;

template <Elem E, typename ACC>
__device__ __forceinline__ ACC mma(u32x4_t a, u32x4_t b, ACC c) {
    if constexpr (E == Elem::bf16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                       c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0,
                                                     0, 0);
}

// One fp32 instruction (`s` of the four a step) for each pair of blocks of a wavefront's first
// `nblk` row blocks.  (The guards, which a full tile falls through, are compared anew each
// time: scalar compares; masks that are kept cost vector instructions.)
template <int FM, int FN>
__device__ __forceinline__ void mma_f32(const u32x4_t (&af)[FM], const u32x4_t (&bf)[FN], int s, f32x4_t (&acc)[FM][FN],
                                        int nblk) {
    if (!__builtin_constant_p(nblk)) asm volatile("" : "+s"(nblk));
#pragma unroll
    for (int i = 0; i < FM; ++i)
        if (__builtin_expect(i < nblk, 1)) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(af[i][s]), __uint_as_float(bf[j][s]),
                                                                 acc[i][j], 0, 0, 0);
        }
}

// One step's products of a wavefront.  fp32 takes four instructions per pair of blocks, which
// follow each other only after every other pair's, so that none waits for the one before it.
template <Elem E, typename ACC, int FM, int FN>
__device__ __forceinline__ void mma_step(const u32x4_t (&af)[FM], const u32x4_t (&bf)[FN], ACC (&acc)[FM][FN], int nblk) {
    if constexpr (E == Elem::f32) {
#pragma unroll
        for (int s = 0; s < 4; ++s) mma_f32(af, bf, s, acc, nblk);
    } else {
        if (!__builtin_constant_p(nblk)) asm volatile("" : "+s"(nblk));
#pragma unroll
        for (int i = 0; i < FM; ++i)
            if (__builtin_expect(i < nblk, 1)) {
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mma<E>(af[i], bf[j], acc[i][j]);
            }
    }
}

// A wavefront's operands of a step, from a stage of the A operand's T_A x 64 bytes, then the
// B operand's.
template <int TA, typename RA, typename RB, int FM, int FN>
__device__ __attribute__((always_inline)) inline void read_stage(const lds_char* __restrict__ rd, int ablk, int bblk,
                                                                 const RA& ra, const RB& rb, u32x4_t (&af)[FM],
                                                                 u32x4_t (&bf)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i) af[i] = ra(rd, ablk + i);
#pragma unroll
    for (int j = 0; j < FN; ++j) bf[j] = rb(rd + TA * 64, bblk + j);
}

// Reads a wavefront's operands of a step from stage `rd` and starts its share of a later
// step's loads into stage `wr`.  The two are separate __restrict__ arguments: otherwise the
// compiler takes the transposing reads to touch what is in flight, and waits for every load
// before them.  W wavefronts share the loads.
template <typename O, int TA, int TB, int W, typename OA, typename OB, typename RA, typename RB, int FM, int FN>
__device__ __attribute__((always_inline)) inline void read_and_load(const lds_char* __restrict__ rd,
                                                                    lds_char* __restrict__ wr, int kt, int ablk, int bblk,
                                                                    int wave, const OA& oa, const OB& ob, const RA& ra,
                                                                    const RB& rb, u32x4_t (&af)[FM], u32x4_t (&bf)[FN]) {
    read_stage<TA>(rd, ablk, bblk, ra, rb, af, bf);
    __builtin_amdgcn_sched_barrier(0);
    oa.load(wr, wave * (TA / 16 / W), kt);
    ob.load(wr + TA * 64, wave * (TB / 16 / W), kt);
}

// Work item of block b of a grid of `grid` blocks.  Workgroups are dealt to the eight XCDs in
// turn; 32 consecutive items go to one XCD, so that the tiles they share meet in its L2.
__device__ __forceinline__ int item_of_block(int b, int grid) {
    return b < (grid & ~255) ? (b & ~255) | ((b & 7) << 5) | ((b >> 3) & 31) : b;
}
// Item `w` of a block of ni x nj tiles: G tile rows together, column by column, so that
// consecutive items share a few row operands and a few column operands.
template <int G = 4>
__device__ __forceinline__ void tile_coords(int w, int ni, int nj, int& i, int& j) {
    const int rg = w / (G * nj), in = min(G, ni - G * rg), l = w - rg * G * nj;
    j = l / in;
    i = G * rg + l % in;
}

// The tile of work item w: its place in C and its two operands.
struct Tile2 {
    int e, i0, ni, j0, nj;        // group; first row (of the rows, kind 2: of the matrix) and rows; first column and columns
    int C;                        // contraction length
    long long crow;               // first row within C
    uint64_t abase, bbase;        // first bytes of the operands
    uint64_t abase2, bbase2;      // of the second ones, where the variant has any
    // steps of the contraction
    template <typename O>
    __device__ __forceinline__ int steps() const { return (C + O::kStep - 1) / O::kStep * (O::kTwo ? 2 : 1); }
};
// Two weight gradients of the same rows in one launch (grid of two rows): the second row's workgroups
// take the second operand and output, so that one's last tiles run beside the other's first.  gated_mm's
// whole gradient, 64 groups, 32768 rows (Zipf), 7168 x 2048 bf16: 4426 -> 4354 us; 24 groups, 4999
// rows, 1032 x 712 fp32: 332 -> 319.
template <typename O>
__device__ __forceinline__ void take_pair(MmArgs& a) {
    if constexpr (O::KIND == 2)
        if (blockIdx.y) {
            a.b = a.b2;
            a.c = a.ca;
        }
}
template <typename O>
unsigned pair_rows(const MmArgs& a) { return O::KIND == 2 && a.b2 ? 2 : 1; }

// columns of C in a tile whose B operand fills BN columns of a stage
template <typename O>
constexpr int tile_cols(int BN) { return O::kGated ? BN / 2 : BN; }

// Work items of a launch (all its tiles); fills `g` and, if asked, zeros the rows of no group.
// Call with all threads.
template <typename O, int BM, int BN, typename OUT>
__device__ __forceinline__ int count_items(const MmArgs& a, Groups& g) {
    const int J = O::KIND == 1 ? a.K : a.N, NJ = (J + BN - 1) / BN;
    if constexpr (O::KIND == 2) {
        return a.E * ((a.K + BM - 1) / BM) * NJ;             // the tiles of every expert's matrix, rows or not
    } else {
        load_groups(a.offsets, a.E, a.rows, BM, g);
        if (a.zero_rest) {
            zero_rest(a.offsets, a.E, a.rows, a.c, (long long)J * sizeof(OUT), blockIdx.x, gridDim.x);
            if constexpr (O::kGated)
                if (a.ca) {
                    zero_rest(a.offsets, a.E, a.rows, a.ca, (long long)J * sizeof(OUT), blockIdx.x, gridDim.x);
                    zero_rest(a.offsets, a.E, a.rows, a.cb, (long long)J * sizeof(OUT), blockIdx.x, gridDim.x);
                }
        }
        return uni(g.pre[a.E]) * NJ;
    }
}

// Tile of work item w.  Group rows are cut evenly: a group of r rows gets ceil(r / BM) tiles
// of about r / tiles rows each, in multiples of 16 (a group a little above a multiple of BM
// then has no nearly empty tile).  64 experts of 256 +- 16 rows, 2048 -> 1408: 180 -> 166 us.
template <typename O, int BM, int BN>
__device__ __forceinline__ void tile_of_item(const MmArgs& a, const Groups& g, int w, Tile2& t) {
    const int J = O::KIND == 1 ? a.K : a.N, NJ = (J + BN - 1) / BN;
    int it, jt, r0, r1;
    if constexpr (O::KIND == 2) {
        const int NI = (a.K + BM - 1) / BM;
        t.e = uni(w / (NI * NJ));
        tile_coords(w - t.e * NI * NJ, NI, NJ, it, jt);
        group_rows(a.offsets, t.e, a.rows, r0, r1);
        r0 = uni(r0);
        r1 = uni(r1);
        t.i0 = uni(it * BM);
        t.j0 = uni(jt * BN);
        t.ni = min(BM, a.K - t.i0);
        t.C = r1 - r0;
        t.crow = (long long)t.e * a.K + t.i0;
        t.abase = (uint64_t)a.a + ((uint64_t)r0 * a.K + t.i0) * O::ES;
        t.bbase = (uint64_t)a.b + ((uint64_t)r0 * a.N + t.j0) * O::ES;
    } else {
        t.e = uni(group_of_tile(g.pre, a.E, w / NJ));
        const int p0 = uni(g.pre[t.e]), tiles = uni(g.pre[t.e + 1]) - p0;
        tile_coords(w - p0 * NJ, tiles, NJ, it, jt);
        r0 = uni(g.r0[t.e]);
        r1 = uni(g.r1[t.e]);
        // (the clamps do nothing for offsets that do not decrease; for others, whose tile counts
        // mean nothing, they keep the tile inside the group and the matrix)
        const int h = min(max(((r1 - r0 + tiles - 1) / max(tiles, 1) + 15) / 16 * 16, 16), BM);
        t.i0 = uni(min(max(r0 + it * h, r0), r1));
        t.j0 = uni(min(max(jt, 0), NJ - 1) * BN);
        t.ni = uni(min(h, r1 - t.i0));
        t.C = O::KIND == 1 ? a.N : a.K;
        t.crow = t.i0;
        t.abase = (uint64_t)a.a + (uint64_t)t.i0 * t.C * O::ES;
        const uint64_t mat = (uint64_t)a.b + (uint64_t)t.e * a.K * a.N * O::ES;
        t.bbase = mat + (O::kBCols ? (uint64_t)t.j0 : (uint64_t)t.j0 * t.C) * O::ES;
    }
    if constexpr (O::kTwo) t.abase2 = uni(t.abase - (uint64_t)a.a + (uint64_t)a.a2);
    if constexpr (O::kTwo || O::kGated) t.bbase2 = uni(t.bbase - (uint64_t)a.b + (uint64_t)a.b2);
    t.abase = uni(t.abase);
    t.bbase = uni(t.bbase);
    t.nj = min(BN, J - t.j0);
}

template <typename O, int T, int N, bool R32 = false>
__device__ __forceinline__ OperandA<O, T, N, R32> operand_a(const MmArgs& a, const Tile2& t) {
    Operand<O::ES, O::kACols, T, N, R32> o;
    o.base = t.abase;
    o.ld = (O::KIND == 2 ? a.K : t.C) * O::ES;
    o.n = O::kACols ? t.C : t.ni;
    o.cbytes = t.C * O::ES;
    if constexpr (O::kTwo) return {o, t.abase2, (t.C + O::kStep - 1) / O::kStep};
    else return o;
}
template <typename O, int T, int N, bool R32 = false>
__device__ __forceinline__ OperandB<O, T, N, R32> operand_b(const MmArgs& a, const Tile2& t) {
    constexpr int TB = O::kGated ? T / 2 : T, NB = O::kGated ? N / 2 : N;      // of one matrix
    Operand<O::ES, O::kBCols, TB, NB, R32> o;
    o.base = t.bbase;
    o.ld = (O::kBCols ? a.N : t.C) * O::ES;
    o.n = O::kBCols ? t.C : t.nj;
    o.cbytes = t.C * O::ES;
    if constexpr (O::kTwo) {
        return {o, t.bbase2, (t.C + O::kStep - 1) / O::kStep};
    } else if constexpr (O::kGated) {
        auto up = o;
        up.base = t.bbase2;
        return {o, up};
    } else {
        return o;
    }
}

// SiLU(a) b, in fp32 (rounded to bf16 or not at all).
template <Elem E>
__device__ __forceinline__ float gated(float a, float b) {
    float s, ns;
    sigmoid<E == Elem::bf16>(a, s, ns);
    return a * s * b;
}

// Workgroups for the tiles of a launch (row tiles are bounded from the row count: the group
// sizes stay on the device; the surplus returns at once).
inline long long mm_blocks(const MmArgs& a, int kind, int BM, int BN) {
    const long long J = kind == 1 ? a.K : a.N, NJ = (J + BN - 1) / BN;
    const long long ni = kind == 2 ? (long long)a.E * ((a.K + BM - 1) / BM)
                                   : ((long long)a.rows + BM - 1) / BM + (a.rows < a.E ? a.rows : a.E);
    return ni * NJ;
}

}  // namespace moe
