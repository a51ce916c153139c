// Grouped products, large tiles: 256 x 256 on the matrix cores, one tile per workgroup
// (mm_tile.h has the kinds, the operand layouts and the loads, mm_large.h the tile's division).
//
// The wavefronts of the upper and of the lower rows (one of each per SIMD) run half a step out
// of phase: while one reads its operands and starts loads, the other's matrix instructions
// run; two barriers a step.  Against steps in which every wavefront does both, woven together,
// with one barrier: x W 862 against 906 us, dy W^T 995 against 1017, x^T dy 890 against 926 (8
// experts, 8192 rows, 4096 x 14336 bf16; 1.12, 0.97 and 1.08 PFLOP/s), int8 504 against 514
// (1.91 PFLOP/s); 4096^3 bf16: 110, 109 and 108 us.  What is left: the last, partial round of
// tiles (dy W^T: 2.25 rounds take three), and a tile's first loads and output, 3 to 4 us.
#include "mm_large.h"

namespace moe {

namespace {

using namespace large;

constexpr int kCS = kT + 8;                   // bf16 per row of the output staging tile
constexpr size_t kLds = (size_t)kT * kCS * 2; // staging tile; the stages (128 KB) lie inside
static_assert(kStages * kStage <= (int)kLds, "the stages fit below the staging tile's end");

// The steps of one of the two wavefront groups.  Between two barriers one group is in its read
// phase (R) and the other in its matrix phase (M):
//   group 0:  R0 | M0 | R1 | M1 | ... | M(KT-1) | (idle)
//   group 1: (idle) | R0 | M0 | R1 | ... | R(KT-1) | M(KT-1)
// R(k) starts the loads of step k + 3 into the stage that held step k - 1, which both groups
// have read by then (each read phase ends with lgkmcnt(0) before its barrier).  Step k + 1 is
// waited for before the barrier that opens group 0's R(k+1): by group 0 at the end of M(k),
// by group 1 at the end of R(k).
template <typename O, int GROUP>
__device__ __attribute__((always_inline)) inline void steps(lds_char* lds, int KT, int nblk, int ablk, int wn, int wave,
                                                            const OpA<O>& oa, const OpB<O>& ob,
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
        asm volatile("" : "+s"(nblk));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (__builtin_expect(i < nblk, 1)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = mma<O::ELEM>(bf[j], af[i], acc[i][j]);
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
    extern __shared__ uint4 smem[];
    __shared__ Groups groups;
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), wm = wave >> 2, wn = wave & 3;
    const int l16 = lane & 15, lq = lane >> 4;

    const int w = item_of_block(blockIdx.x, gridDim.x);
    if (w >= count_items<O, kT, kT, OUT>(a, groups)) return;
    Tile2 t;
    tile_of_item<O, kT, kT>(a, groups, w, t);
    auto oa = operand_a<O, kT, kLoads>(a, t);
    auto ob = operand_b<O, kT, kLoads>(a, t);
    oa.plan(wave * kLoads, lane, t.ni);
    ob.plan(wave * kLoads, lane, t.nj);

    // this wavefront's rows, in 16-row blocks: the tile's, split evenly over the two groups
    const int half = min(128, (t.ni + 31) / 32 * 16), row0 = uni(wm * half);
    const int nblk = uni(max(0, min(half, t.ni - row0) + 15) / 16);
    typename O::Acc acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = typename O::Acc{0, 0, 0, 0};

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
        if (wm == 0) steps<O, 0>(lds, KT, nblk, row0 / 16, wn, wave, oa, ob, ra, rb, acc);
        else steps<O, 1>(lds, KT, nblk, row0 / 16, wn, wave, oa, ob, ra, rb, acc);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // the last loads (zeros) land before LDS is reused
        __syncthreads();
    }

    // The tile: scales (int8), one rounding.  Lane l holds row l & 15 and columns 4 (l >> 4)
    // .. + 3 of each 16 x 16 block; bf16 goes out as whole rows through LDS.
    const int J = O::KIND == 1 ? a.K : a.N;
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(3))) u32x2_t lds_u2;
    f32x4_t wsc[4];
    if constexpr (O::ELEM == Elem::i8)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = wn * 64 + 16 * j + 4 * lq;
            wsc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            if (col < t.nj) wsc[j] = *reinterpret_cast<const f32x4_t*>(a.ws + (long long)t.e * a.N + t.j0 + col);
        }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= nblk) break;
        const int r = row0 + 16 * i + l16;
        float xsc = 1.f;
        if constexpr (O::ELEM == Elem::i8) xsc = r < t.ni ? a.xs[t.i0 + r] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = wn * 64 + 16 * j + 4 * lq;
            f32x4_t x;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                x[v] = (float)acc[i][j][v];
                if constexpr (O::ELEM == Elem::i8) x[v] = x[v] * xsc * wsc[j][v];
            }
            if constexpr (sizeof(OUT) == 2)
                *(lds_u2*)(lds + (r * kCS + col) * 2) = u32x2_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
            else if (r < t.ni && col < t.nj)
                *reinterpret_cast<f32x4_t*>((float*)a.c + (t.crow + r) * J + t.j0 + col) = x;
        }
    }
    if constexpr (sizeof(OUT) == 2) {
        __syncthreads();
        for (int c = tid; c < t.ni * 32; c += 512) {
            const int r = c >> 5, cc = (c & 31) * 8;
            if (cc < t.nj)
                __builtin_nontemporal_store(*(const __attribute__((address_space(3))) u32x4_t*)(lds + (r * kCS + cc) * 2),
                                            reinterpret_cast<u32x4_t*>((bf16_t*)a.c + (t.crow + r) * J + t.j0 + cc));
        }
    }
#endif
}

template <typename O, typename OUT>
hipError_t go(const MmArgs& a, hipStream_t st) {
    hipError_t e = allow_lds<k_mm<O, OUT>>(kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_mm<O, OUT>), dim3((unsigned)mm_blocks(a, O::KIND, kT, kT)), dim3(512), kLds, st, a);
    return hipGetLastError();
}

}  // namespace

// Groups of middling size go in a stream of tiles.  Smaller ones are a matter of writing the
// matrices, which many workgroups at once do better; larger ones of the steps themselves.  Here
// and there, in us: 64 experts, 2048 x 1408, rows a group 32: 85 and 95, 64: 95 and 95, 256: 153
// and 150; 8 experts, 4096 x 4096, 64: 76 and 65; 256 experts, 1024 x 512, 234: 105 and 101; 8
// experts, 4096 x 14336, 1024: 890 and 921.
bool mm_streams(const MmArgs& a) {
    const long long groups = a.rows < a.E ? a.rows : a.E;
    return a.rows >= 48 * groups && a.rows < 640 * groups;
}

hipError_t launch_mm_large(int kind, int out_dtype, const MmArgs& a, hipStream_t st) {
    const bool f = out_dtype == MOE_F32;
    switch (kind) {
        case 0: return go<Op<0, Elem::bf16>, bf16_t>(a, st);
        case 1: return go<Op<1, Elem::bf16>, bf16_t>(a, st);
        case 2:
            if (mm_streams(a)) return launch_mm_stream(out_dtype, a, st);
            return f ? go<Op<2, Elem::bf16>, float>(a, st) : go<Op<2, Elem::bf16>, bf16_t>(a, st);
        default: return f ? go<Op<3, Elem::i8>, float>(a, st) : go<Op<3, Elem::i8>, bf16_t>(a, st);
    }
}

}  // namespace moe
