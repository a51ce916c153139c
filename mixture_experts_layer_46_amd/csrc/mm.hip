// Grouped products, large tiles: 256 x 256 on the matrix cores (mm_tile.h has the kinds, the
// operand layouts and the loads).
//
// Eight wavefronts in two groups of four (one of each per SIMD); a group owns half the
// tile's rows as 128 x 64 wavefront tiles, 128 accumulator registers each.  The groups run
// half a step out of phase: while one reads its operands from LDS and starts the loads of
// a later step, the other's matrix instructions run.  Operands go into four LDS stages,
// three steps ahead; every wavefront issues the same number of loads per step, so one
// constant vmcnt waits for the step that is needed next.
#include "mm_tile.h"

#include <stdlib.h>
namespace moe {

namespace {

constexpr int kT = 256;                       // tile rows and columns
constexpr int kStage = 2 * kT * 64;           // bytes of a step: the A operand, then the B operand
constexpr int kStages = 4;
constexpr int kCS = kT + 8;                   // bf16 per row of the output staging tile
constexpr size_t kLds = (size_t)kT * kCS * 2; // staging tile; the stages (128 KB) lie inside
static_assert(kStages * kStage <= (int)kLds, "the stages fit below the staging tile's end");
constexpr int kLoads = 2;                     // loads of one operand per wavefront and step
constexpr int kVmcnt = 4 * kLoads;            // loads of the two steps after the awaited one

// The steps of one group.  Between two barriers one group is in its read phase (R) and the
// other in its matrix phase (M):
//   group 0:  R0 | M0 | R1 | M1 | ... | M(KT-1) | (idle)
//   group 1: (idle) | R0 | M0 | R1 | ... | R(KT-1) | M(KT-1)
// R(k) starts the loads of step k + 3 into the stage that held step k - 1, which both groups
// have read by then (each read phase ends with lgkmcnt(0) before its barrier).  Step k + 1 is
// waited for before the barrier that opens group 0's R(k+1): by group 0 at the end of M(k),
// by group 1 at the end of R(k).
template <typename O, int GROUP>
__device__ __attribute__((always_inline)) inline void steps(lds_char* lds, int KT, int nblk, int ablk, int wn, int wave,
                                                            const Operand<O::ES, O::kACols, kT, kLoads>& oa,
                                                            const Operand<O::ES, O::kBCols, kT, kLoads>& ob,
                                                            const Reader<O::ES, O::kACols, kT>& ra,
                                                            const Reader<O::ES, O::kBCols, kT>& rb,
                                                            typename O::Acc (&acc)[8][4]) {
    u32x4_t af[8], bf[4];
    if constexpr (GROUP == 1) lds_barrier();
    for (int kt = 0; kt < KT; ++kt) {
        read_and_load<O, kT, kT, 8>(lds + (kt % kStages) * kStage, lds + ((kt + 3) % kStages) * kStage, kt + 3, ablk, wn * 4,
                                    wave, oa, ob, ra, rb, af, bf);
        wait_lds();
        if constexpr (GROUP == 1) wait_vmcnt<kVmcnt>();
        lds_barrier();
        // a full tile falls through the guards
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (__builtin_expect(i < nblk, 1)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = mma<O::ELEM>(af[i], bf[j], acc[i][j]);
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

template <typename O, typename OUT>
__global__ __launch_bounds__(512, 1) void k_mm(MmArgs a) {
#ifdef __HIP_DEVICE_COMPILE__          // the host pass needs the signature only
    using ACC = typename O::Acc;
    extern __shared__ uint4 smem[];
    __shared__ int pre[257];
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int grp = wave >> 2, wn = wave & 3, l16 = lane & 15, lq = lane >> 4;

    Tile2 t;
    if (!find_tile<O, kT, kT, OUT>(a, pre, t)) return;
    auto oa = operand_a<O, kT, kLoads>(a, t);
    auto ob = operand_b<O, kT, kLoads>(a, t);
    oa.plan(wave * kLoads, lane, t.ni);
    ob.plan(wave * kLoads, lane, t.nj);

    // rows split evenly over the two groups, in 16-row blocks
    const int half = min(128, (t.ni + 31) / 32 * 16), row0 = grp * half;
    const int nblk = max(0, min(half, t.ni - row0) + 15) / 16;
    ACC acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = ACC{0, 0, 0, 0};

    const int KT = (t.C + O::kStep - 1) / O::kStep;
    if (KT > 0) {
        const Reader<O::ES, O::kACols, kT> ra(lane);
        const Reader<O::ES, O::kBCols, kT> rb(lane);
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            oa.load(lds + s * kStage, wave * kLoads, s);
            ob.load(lds + s * kStage + kT * 64, wave * kLoads, s);
        }
        wait_vmcnt<kVmcnt>();
        lds_barrier();
        if (grp == 0) steps<O, 0>(lds, KT, nblk, row0 / 16, wn, wave, oa, ob, ra, rb, acc);
        else steps<O, 1>(lds, KT, nblk, row0 / 16, wn, wave, oa, ob, ra, rb, acc);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the last loads (zeros) land before LDS is reused
        __syncthreads();
    }

    // epilogue: scales (int8), one rounding, whole rows through LDS
    const int J = O::KIND == 1 ? a.K : a.N;
    float wsc[4] = {1.f, 1.f, 1.f, 1.f};
    if constexpr (O::ELEM == Elem::i8)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = wn * 64 + 16 * j + l16;
            wsc[j] = col < t.nj ? a.ws[(long long)t.e * a.N + t.j0 + col] : 0.f;
        }
    typedef __attribute__((address_space(3))) bf16_t lds_bf16;
    lds_bf16* sC = reinterpret_cast<lds_bf16*>(lds);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= nblk) break;
        const int r = row0 + 16 * i + 4 * lq;
        float xsc[4] = {1.f, 1.f, 1.f, 1.f};
        if constexpr (O::ELEM == Elem::i8)
#pragma unroll
            for (int v = 0; v < 4; ++v) xsc[v] = a.xs[t.i0 + min(r + v, t.ni - 1)];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = wn * 64 + 16 * j + l16;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                float val = (float)acc[i][j][v];
                if constexpr (O::ELEM == Elem::i8) val = val * xsc[v] * wsc[j];
                if constexpr (sizeof(OUT) == 2) {
                    sC[(r + v) * kCS + col] = f32_to_bf16(val);
                } else {
                    if (r + v < t.ni && col < t.nj) ((float*)a.c)[(t.crow + r + v) * J + t.j0 + col] = val;
                }
            }
        }
    }
    if constexpr (sizeof(OUT) == 2) {
        __syncthreads();
        for (int c = tid; c < t.ni * 32; c += 512) {
            const int r = c >> 5, cc = (c & 31) * 8;
            if (cc < t.nj)
                __builtin_nontemporal_store(
                    *reinterpret_cast<const __attribute__((address_space(3))) u32x4_t*>(sC + r * kCS + cc),
                    reinterpret_cast<u32x4_t*>((bf16_t*)a.c + (t.crow + r) * J + t.j0 + cc));
        }
    }
#endif
}

template <typename O, typename OUT>
hipError_t go(const MmArgs& a, hipStream_t st) {
    auto kern = k_mm<O, OUT>;
    hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)mm_blocks(a, O::KIND, kT, kT)), dim3(512), kLds, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mm_large(int kind, int out_dtype, const MmArgs& a, hipStream_t st) {
    const bool f = out_dtype == MOE_F32;
    switch (kind) {
        case 0: return go<Op<0, Elem::bf16>, bf16_t>(a, st);
        case 1: return go<Op<1, Elem::bf16>, bf16_t>(a, st);
        case 2: return f ? go<Op<2, Elem::bf16>, float>(a, st) : go<Op<2, Elem::bf16>, bf16_t>(a, st);
        default: return f ? go<Op<3, Elem::i8>, float>(a, st) : go<Op<3, Elem::i8>, bf16_t>(a, st);
    }
}


hipError_t launch_mm(int kind, int dtype, int out_dtype, const MmArgs& a, hipStream_t st) {
    // TUNING
    const char* f = getenv("MM_FORM");
    if (f) {
        if (f[0] == 'L' && (dtype == MOE_BF16 || kind == 3)) return launch_mm_large(kind, out_dtype, a, st);
        if (f[0] == 'M') return launch_mm_mid(atoi(f + 1), kind, dtype, out_dtype, a, st);
        if (f[0] == 'T' && kind != 2) return launch_mm_thin(atoi(f + 2), f[1] - '0', kind, dtype, out_dtype, a, st);
    }
    if (dtype == MOE_F32 && kind != 3) return launch_mm_mid(128, kind, dtype, out_dtype, a, st);
    return launch_mm_large(kind, out_dtype, a, st);
}

}  // namespace moe
