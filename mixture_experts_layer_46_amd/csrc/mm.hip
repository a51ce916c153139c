// Grouped products on the matrix cores (bf16 with fp32 sums, and int8 with int32 sums).
//
//   kind 0  y[r, n]     = sum_k x[r, k] w[e, k, n]     (rows r of group e)
//   kind 1  dx[r, k]    = sum_n dy[r, n] w[e, k, n]
//   kind 2  dw[e, k, n] = sum_r x[r, k] dy[r, n]       (r over the rows of group e)
//   kind 3  y[r, n]     = (sum_k xq[r, k] wq[e, n, k]) xs[r] ws[e, n]
//
// All four are C[i, j] = sum_c A[i, c] B[c, j] on 256 x 256 tiles, with each operand in one
// of two layouts in memory:
//   rows      the contraction index runs along memory (x, dy, and wq; w for kind 1).  In LDS
//             a row keeps one step of 64 bytes (32 bf16 or 64 int8) as four 16-byte chunks,
//             chunk q of row m at q ^ swa4(m); a matrix operand is one ds_read_b128.
//   columns   the tile index runs along memory (w for kind 0; both operands of kind 2).  In
//             LDS a step is 32 rows of 512 bytes, 16-byte chunk c of row k at c ^ fk(k); a
//             matrix operand (8 consecutive k of one column per lane) is two
//             ds_read_b64_tr_b16.
// The 16x16x32 bf16 and the 16x16x64 int8 instruction take the same bytes per lane and the
// same time, so kinds 1 and 3 are one kernel but for the instruction and the epilogue.
//
// Eight wavefronts in two groups of four (one of each per SIMD); a group owns half the
// tile's rows as 128 x 64 wavefront tiles, 128 accumulator registers each.  The groups run
// half a step out of phase: while one reads its operands from LDS and starts the loads of
// a later step, the other's matrix instructions run.  Operands travel from memory straight
// into four LDS stages, three steps ahead; every wavefront issues the same number of loads
// per step, so one constant vmcnt waits for the step that is needed next.
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "mm_common.h"
#include "mm_launch.h"

namespace moe {

namespace {

typedef short v4i16_t __attribute__((ext_vector_type(4)));
typedef short v8i16_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kT = 256;                       // tile rows and columns
constexpr int kStage = 16384;                 // bytes of one operand's step
constexpr int kStages = 4;
constexpr int kRowB = 64;                     // bytes of one row of a `rows` step
constexpr int kColB = 512;                    // bytes of one row of a `columns` step
constexpr int kBRing = kStages * kStage;
constexpr int kCS = kT + 8;                   // bf16 per row of the output staging tile
constexpr size_t kLds = (size_t)kT * kCS * 2; // staging tile; the rings (128 KB) lie inside
static_assert(2 * kBRing <= (int)kLds, "the rings fit below the staging tile's end");
constexpr int kVmcnt = 8;                     // loads of the two steps after the awaited one

__device__ __forceinline__ void lds_barrier() { asm volatile("s_barrier" ::: "memory"); }
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }      // lgkmcnt(0)
__device__ __forceinline__ int fk(int k) { return 2 * ((k & 3) | (((k >> 3) & 1) << 2)); }

template <int KIND>
struct Kind {
    static constexpr bool kACols = KIND == 2, kBCols = KIND == 0 || KIND == 2, kInt8 = KIND == 3;
    static constexpr int kStepC = kInt8 ? 64 : 32;       // contraction indexes per step
    static constexpr int kElem = kInt8 ? 1 : 2;
};

// One operand of one tile: what a wavefront needs to start the loads of a step.  Loads of
// rows or columns past the tile, and of contraction indexes past the end, read zeros (an
// offset past the buffer's end).
template <bool COLS>
struct Operand {
    uint64_t base;            // tile's first row (rows), or its first contraction row (columns)
    uint32_t ld;              // bytes from one memory row to the next
    uint32_t rows;            // rows: valid tile rows; columns: contraction length
    uint32_t cbytes;          // rows: bytes of the contraction
    uint32_t off[2];          // this lane's offset of its two loads, at step 0
    uint32_t kq;              // rows: this lane's byte within the step

    // `valid`: rows: rows of the tile that exist; columns: columns that exist
    __device__ __forceinline__ void plan(int wave, int lane, int valid) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = wave * 2 + i;
            if constexpr (COLS) {
                const int k = j * 2 + (lane >> 5), c = (lane & 31) ^ fk(k);
                off[i] = 8 * c < valid ? (uint32_t)k * ld + (uint32_t)c * 16 : kOOB;
            } else {
                const int r = j * 16 + (lane >> 2), q = (lane & 3) ^ swa4(r);
                kq = (uint32_t)q * 16;
                off[i] = r < valid ? (uint32_t)r * ld + kq : kOOB;
            }
        }
    }
    __device__ __forceinline__ void load(lds_char* stage, int wave, int kt) const {
        if constexpr (COLS) {
            const int left = (int)rows - kt * 32;
            const uint32_t n = (uint32_t)(left < 0 ? 0 : left > 32 ? 32 : left) * ld;
            const __amdgpu_buffer_rsrc_t r = make_rsrc((const void*)(base + (uint64_t)kt * 32 * ld), n);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(stage + (wave * 2 + i) * 1024), 16, off[i], 0, 0, 0);
        } else {
            const uint32_t k0 = (uint32_t)kt * kRowB;
            const __amdgpu_buffer_rsrc_t r = make_rsrc((const void*)base, rows * ld);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(stage + (wave * 2 + i) * 1024), 16,
                                                         (k0 + kq < cbytes && off[i] != kOOB) ? off[i] + k0 : kOOB, 0, 0, 0);
        }
    }
};

// 16-index block `blk` of an operand's step as a matrix operand: lane l holds index l & 15
// and the 16 bytes of contraction number l >> 4.
template <bool COLS>
struct Reader {
    int rd, g;
    __device__ __forceinline__ explicit Reader(int lane) {
        const int l16 = lane & 15, lq = lane >> 4;
        if constexpr (COLS) {
            g = ((l16 >> 2) & 3) | ((lq & 1) << 2);
            rd = (8 * lq + (l16 >> 2)) * kColB + (((l16 & 3) >> 1) << 4) + ((l16 & 1) << 3);
        } else {
            g = 0;
            rd = l16 * kRowB + ((lq ^ swa4(l16)) << 4);
        }
    }
    __device__ __forceinline__ u32x4_t operator()(const lds_char* stage, int blk) const {
        if constexpr (COLS) {
            const lds_char* p = stage + rd + (((blk & ~7) | ((blk & 7) ^ g)) << 5);
            const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16_t*)p);
            const v4i16_t hi =
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16_t*)(p + 4 * kColB));
            const v8i16_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            return __builtin_bit_cast(u32x4_t, v);
        } else {
            return *(const __attribute__((address_space(3))) u32x4_t*)(stage + rd + blk * 16 * kRowB);
        }
    }
};

__device__ __forceinline__ f32x4_t mma(u32x4_t a, u32x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}
__device__ __forceinline__ i32x4_t mma(u32x4_t a, u32x4_t b, i32x4_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0,
                                                 0);
}

// The steps of one group.  Between two barriers one group is in its read phase (R) and the
// other in its matrix phase (M):
//   group 0:  R0 | M0 | R1 | M1 | ... | M(KT-1) | (idle)
//   group 1: (idle) | R0 | M0 | R1 | ... | R(KT-1) | M(KT-1)
// R(k) starts the loads of step k + 3 into the stage that held step k - 1, which both groups
// have read by then (each read phase ends with lgkmcnt(0) before its barrier).  Step k + 1 is
// waited for before the barrier that opens group 0's R(k+1): by group 0 at the end of M(k),
// by group 1 at the end of R(k).
template <int KIND, int GROUP, typename ACC>
__device__ __attribute__((always_inline)) inline void steps(lds_char* lds, int KT, int nblk, int ablk, int wn, int wave,
                                                            const Operand<Kind<KIND>::kACols>& oa,
                                                            const Operand<Kind<KIND>::kBCols>& ob,
                                                            const Reader<Kind<KIND>::kACols>& ra,
                                                            const Reader<Kind<KIND>::kBCols>& rb, ACC (&acc)[8][4]) {
    u32x4_t af[8], bf[4];
    if constexpr (GROUP == 1) lds_barrier();
    for (int kt = 0; kt < KT; ++kt) {
        const lds_char *as = lds + (kt % kStages) * kStage, *bs = as + kBRing;
#pragma unroll
        for (int i = 0; i < 8; ++i) af[i] = ra(as, ablk + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) bf[i] = rb(bs, wn * 4 + i);
        __builtin_amdgcn_sched_barrier(0);
        lds_char* ns = lds + ((kt + 3) % kStages) * kStage;
        oa.load(ns, wave, kt + 3);
        ob.load(ns + kBRing, wave, kt + 3);
        wait_lds();
        if constexpr (GROUP == 1) wait_vmcnt<kVmcnt>();
        lds_barrier();
        // a full tile falls through the guards
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (__builtin_expect(i < nblk, 1)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = mma(af[i], bf[j], acc[i][j]);
            }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[i][j]));
        if constexpr (GROUP == 0) wait_vmcnt<kVmcnt>();
        lds_barrier();
    }
    if constexpr (GROUP == 0) lds_barrier();
}

// Work item of a workgroup.  Workgroups are dealt to the eight XCDs in turn; 32 consecutive
// items go to one XCD, so that the tiles they share meet in its L2.
__device__ __forceinline__ int item_of_block(int b, int grid) {
    return b < (grid & ~255) ? (b & ~255) | ((b & 7) << 5) | ((b >> 3) & 31) : b;
}
// Item `w` of a block of ni x nj tiles: four tile rows together, column by column, so that 32
// consecutive items share 4 row operands and 8 column operands.
__device__ __forceinline__ void tile_coords(int w, int ni, int nj, int& i, int& j) {
    const int rg = w / (4 * nj), in = min(4, ni - 4 * rg), l = w - rg * 4 * nj;
    j = l / in;
    i = 4 * rg + l % in;
}

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uni(uint64_t v) {
    return ((uint64_t)(uint32_t)uni((int)(v >> 32)) << 32) | (uint32_t)uni((int)(uint32_t)v);
}

template <int KIND, typename OUT>
__global__ __launch_bounds__(512, 1) void k_mm(MmArgs a) {
    using S = Kind<KIND>;
    using ACC = std::conditional_t<S::kInt8, i32x4_t, f32x4_t>;
    extern __shared__ uint4 smem[];
    __shared__ int pre[257];
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int grp = wave >> 2, wn = wave & 3, l16 = lane & 15, lq = lane >> 4;

    // ---- which tile
    const int J = KIND == 1 ? a.K : a.N, NJ = (J + kT - 1) / kT;
    const int w = item_of_block(blockIdx.x, gridDim.x);
    int e, i0, ni, jt, C;                                 // group, first output row, rows, column tile, contraction
    long long crow;                                       // first output row within C
    Operand<S::kACols> oa;
    Operand<S::kBCols> ob;
    if constexpr (KIND == 2) {
        const int NI = (a.K + kT - 1) / kT;
        e = w / (NI * NJ);
        int it, r0, r1;
        tile_coords(w - e * NI * NJ, NI, NJ, it, jt);
        group_rows(a.offsets, e, a.rows, r0, r1);
        i0 = it * kT;
        ni = min(kT, a.K - i0);
        C = uni(r1 - r0);
        crow = (long long)e * a.K + i0;
        oa.base = (uint64_t)a.a + ((uint64_t)r0 * a.K + i0) * 2;
        oa.ld = a.K * 2;
        oa.rows = C;
        ob.base = (uint64_t)a.b + ((uint64_t)r0 * a.N + jt * kT) * 2;
        ob.ld = a.N * 2;
        ob.rows = C;
    } else {
        build_row_tiles(a.offsets, a.E, a.rows, kT, pre);
        if (a.zero_rest) zero_rest(a.offsets, a.E, a.rows, a.c, (long long)J * sizeof(OUT), blockIdx.x, gridDim.x);
        const int total = pre[a.E];
        if ((long long)w >= (long long)total * NJ) return;
        e = group_of_tile(pre, a.E, w / NJ);
        int it, r0, r1;
        tile_coords(w - pre[e] * NJ, pre[e + 1] - pre[e], NJ, it, jt);
        group_rows(a.offsets, e, a.rows, r0, r1);
        i0 = r0 + it * kT;
        ni = min(kT, r1 - i0);
        C = KIND == 1 ? a.N : a.K;
        crow = i0;
        oa.ld = C * S::kElem;
        oa.base = (uint64_t)a.a + (uint64_t)i0 * oa.ld;
        oa.rows = uni(ni);
        oa.cbytes = oa.ld;
        const uint64_t mat = (uint64_t)a.b + (uint64_t)e * a.K * a.N * S::kElem;
        if constexpr (S::kBCols) {
            ob.ld = a.N * 2;
            ob.base = mat + (uint64_t)jt * kT * 2;
            ob.rows = C;
        } else {
            ob.ld = C * S::kElem;
            ob.base = mat + (uint64_t)jt * kT * ob.ld;
            ob.rows = uni(min(kT, J - jt * kT));
            ob.cbytes = ob.ld;
        }
    }
    oa.base = uni(oa.base);
    ob.base = uni(ob.base);
    e = uni(e), ni = uni(ni), jt = uni(jt);
    const int j0 = jt * kT, nj = min(kT, J - j0);
    oa.plan(wave, lane, ni);
    ob.plan(wave, lane, nj);

    // ---- rows split evenly over the two groups, in 16-row blocks
    const int half = min(128, (ni + 31) / 32 * 16), row0 = grp * half;
    const int nblk = max(0, min(half, ni - row0) + 15) / 16;
    ACC acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = ACC{0, 0, 0, 0};

    const int KT = (C + S::kStepC - 1) / S::kStepC;
    if (KT > 0) {
        const Reader<S::kACols> ra(lane);
        const Reader<S::kBCols> rb(lane);
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            oa.load(lds + s * kStage, wave, s);
            ob.load(lds + s * kStage + kBRing, wave, s);
        }
        wait_vmcnt<kVmcnt>();
        lds_barrier();
        if (grp == 0) steps<KIND, 0>(lds, KT, nblk, row0 / 16, wn, wave, oa, ob, ra, rb, acc);
        else steps<KIND, 1>(lds, KT, nblk, row0 / 16, wn, wave, oa, ob, ra, rb, acc);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the last loads (zeros) land before LDS is reused
        __syncthreads();
    }

    // ---- epilogue
    float wsc[4] = {1.f, 1.f, 1.f, 1.f};
    if constexpr (S::kInt8)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = wn * 64 + 16 * j + l16;
            wsc[j] = col < nj ? a.ws[(long long)e * a.N + j0 + col] : 0.f;
        }
    typedef __attribute__((address_space(3))) bf16_t lds_bf16;
    lds_bf16* sC = reinterpret_cast<lds_bf16*>(lds);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= nblk) break;
        const int r = row0 + 16 * i + 4 * lq;
        float xsc[4] = {1.f, 1.f, 1.f, 1.f};
        if constexpr (S::kInt8)
#pragma unroll
            for (int v = 0; v < 4; ++v) xsc[v] = a.xs[i0 + min(r + v, ni - 1)];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = wn * 64 + 16 * j + l16;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                float val = (float)acc[i][j][v];
                if constexpr (S::kInt8) val = val * xsc[v] * wsc[j];
                if constexpr (sizeof(OUT) == 2) {
                    sC[(r + v) * kCS + col] = f32_to_bf16(val);
                } else {
                    if (r + v < ni && col < nj) ((float*)a.c)[(crow + r + v) * J + j0 + col] = val;
                }
            }
        }
    }
    if constexpr (sizeof(OUT) == 2) {
        __syncthreads();
        for (int c = tid; c < ni * 32; c += 512) {
            const int r = c >> 5, cc = (c & 31) * 8;
            if (cc < nj)
                __builtin_nontemporal_store(
                    *reinterpret_cast<const __attribute__((address_space(3))) u32x4_t*>(sC + r * kCS + cc),
                    reinterpret_cast<u32x4_t*>((bf16_t*)a.c + (crow + r) * J + j0 + cc));
        }
    }
}

template <int KIND, typename OUT>
hipError_t go(const MmArgs& a, hipStream_t st) {
    auto kern = k_mm<KIND, OUT>;
    hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)kLds);
    if (e != hipSuccess) return e;
    const int J = KIND == 1 ? a.K : a.N, NJ = (J + kT - 1) / kT;
    const long long tiles = KIND == 2 ? (long long)a.E * ((a.K + kT - 1) / kT)
                                      : ((long long)a.rows + kT - 1) / kT + (a.rows < a.E ? a.rows : a.E);
    hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * NJ)), dim3(512), kLds, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mm(int kind, int out_dtype, const MmArgs& a, hipStream_t st) {
    const bool f = out_dtype == MOE_F32;
    switch (kind) {
        case 0: return go<0, bf16_t>(a, st);
        case 1: return go<1, bf16_t>(a, st);
        case 2: return f ? go<2, float>(a, st) : go<2, bf16_t>(a, st);
        default: return f ? go<3, float>(a, st) : go<3, bf16_t>(a, st);
    }
}

}  // namespace moe
