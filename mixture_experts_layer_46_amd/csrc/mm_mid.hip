// Grouped products, tiles of 64 and 128: for groups or matrices too small to fill the chip
// with 256 x 256 tiles, and for fp32 (mm_tile.h has the kinds, layouts and loads).
//
// Four wavefronts, 2 x 2 over the tile; S stages in LDS with the loads S - 1 steps ahead and
// one barrier per step: a wavefront that passes step k's barrier has finished step k - 1,
// whose stage the loads of step k + S - 1 then fill.  Two or more workgroups share a CU and
// cover each other's waits, where the large kernel needs its two groups.
//
// fp32 runs the 16x16x4 instruction, at the card's full fp32 rate; its operands cost a
// fraction of the time that the instructions take, so nothing else is done for it.
#include "mm_tile.h"

namespace moe {

namespace {

template <typename O, int BM, int BN, int S>
struct Mid {
    static constexpr int FM = BM / 32, FN = BN / 32;          // 16-index blocks of a wavefront
    static constexpr int NA = BM / 64, NB = BN / 64;          // loads per wavefront and step
    static constexpr int kA = BM * 64, kStage = (BM + BN) * 64;
    static constexpr int kCS = BN + 8;                        // bf16 per row of the staging tile
    static constexpr size_t kOut = (size_t)BM * kCS * 2;
    static constexpr size_t kLds = kOut > (size_t)S * kStage ? kOut : (size_t)S * kStage;
};

template <typename O, int BM, int BN, int S, typename OUT>
__global__ __launch_bounds__(256, 2) void k_mm_mid(MmArgs a) {
#ifdef __HIP_DEVICE_COMPILE__          // the host pass needs the signature only
    using L = Mid<O, BM, BN, S>;
    using ACC = typename O::Acc;
    extern __shared__ uint4 smem[];
    __shared__ Groups groups;
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1, l16 = lane & 15, lq = lane >> 4;

    Tile2 t;
    const int w = item_of_block(blockIdx.x, gridDim.x);
    if (w >= count_items<O, BM, BN, OUT>(a, groups)) return;
    tile_of_item<O, BM, BN>(a, groups, w, t);
    auto oa = operand_a<O, BM, L::NA>(a, t);
    auto ob = operand_b<O, BN, L::NB>(a, t);
    oa.plan(wave * L::NA, lane, t.ni);
    ob.plan(wave * L::NB, lane, t.nj);
    const Reader<O::ES, O::kACols, BM> ra(lane);
    const Reader<O::ES, O::kBCols, BN> rb(lane);

    // rows split evenly over the two wavefront rows, in 16-row blocks
    const int half = min(BM / 2, (t.ni + 31) / 32 * 16), row0 = wm * half;
    const int nblk = max(0, min(half, t.ni - row0) + 15) / 16;
    ACC acc[L::FM][L::FN];
#pragma unroll
    for (int i = 0; i < L::FM; ++i)
#pragma unroll
        for (int j = 0; j < L::FN; ++j) acc[i][j] = ACC{0, 0, 0, 0};

    const int KT = (t.C + O::kStep - 1) / O::kStep;
    if (KT > 0) {
#pragma unroll
        for (int s = 0; s < S - 1; ++s) {
            oa.load(lds + s * L::kStage, wave * L::NA, s);
            ob.load(lds + s * L::kStage + L::kA, wave * L::NB, s);
        }
        int st = 0, nx = S - 1;                               // stage of this step, and of the loads it starts
        for (int kt = 0; kt < KT; ++kt) {
            wait_vmcnt<(S - 2) * (L::NA + L::NB)>();
            lds_barrier();
            u32x4_t af[L::FM], bf[L::FN];
            read_and_load<O, BM, BN, 4>(lds + st * L::kStage, lds + nx * L::kStage, kt + S - 1, row0 / 16, wn * L::FN, wave, oa,
                                     ob, ra, rb, af, bf);
            wait_lds();
            mma_step<O::ELEM>(af, bf, acc, nblk);
            st = st + 1 == S ? 0 : st + 1;
            nx = nx + 1 == S ? 0 : nx + 1;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // the last loads (zeros) land before LDS is reused
        __syncthreads();
    }

    const int J = O::KIND == 1 ? a.K : a.N;
    float wsc[L::FN];
    if constexpr (O::ELEM == Elem::i8)
#pragma unroll
        for (int j = 0; j < L::FN; ++j) {
            const int col = wn * (BN / 2) + 16 * j + l16;
            wsc[j] = col < t.nj ? a.ws[(long long)t.e * a.N + t.j0 + col] : 0.f;
        }
    typedef __attribute__((address_space(3))) bf16_t lds_bf16;
    lds_bf16* sC = reinterpret_cast<lds_bf16*>(lds);
#pragma unroll
    for (int i = 0; i < L::FM; ++i) {
        if (i >= nblk) break;
        const int r = row0 + 16 * i + 4 * lq;
        float xsc[4];
        if constexpr (O::ELEM == Elem::i8)
#pragma unroll
            for (int v = 0; v < 4; ++v) xsc[v] = a.xs[t.i0 + min(r + v, t.ni - 1)];
#pragma unroll
        for (int j = 0; j < L::FN; ++j) {
            const int col = wn * (BN / 2) + 16 * j + l16;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                float val = (float)acc[i][j][v];
                if constexpr (O::ELEM == Elem::i8) val = val * xsc[v] * wsc[j];
                if constexpr (sizeof(OUT) == 2) {
                    sC[(r + v) * L::kCS + col] = f32_to_bf16(val);
                } else {
                    if (r + v < t.ni && col < t.nj) ((float*)a.c)[(t.crow + r + v) * J + t.j0 + col] = val;
                }
            }
        }
    }
    if constexpr (sizeof(OUT) == 2) {
        __syncthreads();
        constexpr int CPR = BN / 8;
        for (int c = tid; c < t.ni * CPR; c += 256) {
            const int r = c / CPR, cc = (c % CPR) * 8;
            if (cc < t.nj)
                __builtin_nontemporal_store(
                    *reinterpret_cast<const __attribute__((address_space(3))) u32x4_t*>(sC + r * L::kCS + cc),
                    reinterpret_cast<u32x4_t*>((bf16_t*)a.c + (t.crow + r) * J + t.j0 + cc));
        }
    }
#endif
}

template <typename O, int BM, int BN, int S, typename OUT>
hipError_t go(const MmArgs& a, hipStream_t st) {
    constexpr size_t lds = Mid<O, BM, BN, S>::kLds;
    hipError_t e = allow_lds<k_mm_mid<O, BM, BN, S, OUT>>(lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_mm_mid<O, BM, BN, S, OUT>), dim3((unsigned)mm_blocks(a, O::KIND, BM, BN)), dim3(256), lds, st, a);
    return hipGetLastError();
}

template <int BM, int BN, int S>
hipError_t go_kind(int kind, int dtype, int out_dtype, const MmArgs& a, hipStream_t st) {
    const bool f = out_dtype == MOE_F32;
    if (kind == 3) return f ? go<Op<3, Elem::i8>, BM, BN, S, float>(a, st) : go<Op<3, Elem::i8>, BM, BN, S, bf16_t>(a, st);
    if (dtype == MOE_F32)
        return kind == 0   ? go<Op<0, Elem::f32>, BM, BN, S, float>(a, st)
               : kind == 1 ? go<Op<1, Elem::f32>, BM, BN, S, float>(a, st)
                           : go<Op<2, Elem::f32>, BM, BN, S, float>(a, st);
    if (kind == 2) return f ? go<Op<2, Elem::bf16>, BM, BN, S, float>(a, st) : go<Op<2, Elem::bf16>, BM, BN, S, bf16_t>(a, st);
    return kind == 0 ? go<Op<0, Elem::bf16>, BM, BN, S, bf16_t>(a, st) : go<Op<1, Elem::bf16>, BM, BN, S, bf16_t>(a, st);
}

}  // namespace

hipError_t launch_mm_mid(int tile, int kind, int dtype, int out_dtype, const MmArgs& a, hipStream_t st) {
    return tile == 64 ? go_kind<64, 64, 4>(kind, dtype, out_dtype, a, st) : go_kind<128, 128, 4>(kind, dtype, out_dtype, a, st);
}

}  // namespace moe
