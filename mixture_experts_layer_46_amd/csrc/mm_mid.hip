// Grouped products, tiles of 64 and 128: for groups or matrices too small to fill the chip
// with 256 x 256 tiles, and for fp32 (mm_tile.h has the kinds, layouts and loads).
//
// Four wavefronts, 2 x 2 over the tile; S stages of U steps in LDS and one barrier per stage.
// Two or more workgroups share a CU and cover each other's waits, where the large kernel needs
// its two groups.
//
// 16 and 8 bits: loads S - 1 stages ahead; a wavefront that passes a stage's barrier has
// finished the stage before, which the loads then fill.  A workgroup alone on its CU runs at
// the length of its own chain (barrier, LDS reads, products, addresses: some 400 cycles a
// step, the same with every load out of range); reading a step ahead into a second set of
// registers lost 2 to 15% with several workgroups a CU and won 5% at best with one.
//
// fp32 runs the 16x16x4 instruction, at the card's full fp32 rate, and reads a step ahead (3 to
// 7% there).  Beside that instruction every vector instruction counts: the two never overlap
// (matrix and vector cycles together made up 91% of all cycles, whatever else changed), so
// stages are constants of an unrolled loop, operand resources and row guards scalar.  4096
// rows, 2048 x 2048: 292 -> 255 us (dw 306 -> 250, 137 TFLOP/s); 24 groups of 203 rows on
// average, 1032 x 712: 104 -> 92 (dx 94 -> 81, dw 98 -> 87), a single round of tiles, which
// starts and ends with idle matrix units.
#include "mm_tile.h"

namespace moe {

namespace {

template <typename O, int BM, int BN, int S, int U>
struct Mid {
    static constexpr int FM = BM / 32, FN = BN / 32;          // 16-index blocks of a wavefront
    static constexpr int NA = BM / 64, NB = BN / 64;          // loads per wavefront and step
    static constexpr int kSub = (BM + BN) * 64, kStage = U * kSub;      // bytes of one step; of a stage
    static constexpr int kCols = tile_cols<O>(BN);            // columns of C
    static constexpr int kCS = kCols + 8;                     // bf16 per row of the staging tile
    static constexpr size_t kOut = (size_t)BM * kCS * 2;
    static constexpr size_t kLds = kOut > (size_t)S * kStage ? kOut : (size_t)S * kStage;
};

// One fp32 step: the products of the operands in registers, with the next step's read from
// stage `rd` after the first and a later step's loads started into stage `wr` after the second
// of the four instructions per pair of blocks (stages as separate arguments: see read_and_load).
template <typename O, int BM, int BN, int S, typename OA, typename OB, typename RA, typename RB, int FM, int FN>
__device__ __attribute__((always_inline)) inline void step_f32(const lds_char* __restrict__ rd, lds_char* __restrict__ wr,
                                                               int kload, int nblk, int ablk, int bblk, int wave,
                                                               const OA& oa, const OB& ob, const RA& ra, const RB& rb,
                                                               const u32x4_t (&af)[FM], const u32x4_t (&bf)[FN],
                                                               u32x4_t (&an)[FM], u32x4_t (&bn)[FN],
                                                               f32x4_t (&acc)[FM][FN]) {
    constexpr int NA = BM / 64, NB = BN / 64;
    wait_lds();                               // this step's operands are in registers: their stage is free
    wait_vmcnt<(S - 2) * (NA + NB)>();        // this wavefront's loads of the next step have landed
    lds_barrier();                            // everyone's
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        mma_f32(af, bf, s, acc, nblk);
        if (s == 0) read_stage<BM>(rd, ablk, bblk, ra, rb, an, bn);
        if (s == 1) {
            oa.load(wr, wave * NA, kload);
            ob.load(wr + BM * 64, wave * NB, kload);
        }
    }
}

template <typename O, int BM, int BN, int S, int U, typename OUT>
__global__ __launch_bounds__(256, 2) void k_mm_mid(MmArgs a) {
#ifdef __HIP_DEVICE_COMPILE__          // the host pass needs the signature only
    using L = Mid<O, BM, BN, S, U>;
    using ACC = typename O::Acc;
    extern __shared__ uint4 smem[];
    __shared__ Groups groups;
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1, l16 = lane & 15, lq = lane >> 4;

    take_pair<O>(a);
    Tile2 t;
    const int w = item_of_block(blockIdx.x, gridDim.x);
    if (w >= count_items<O, BM, L::kCols, OUT>(a, groups)) return;
    tile_of_item<O, BM, L::kCols>(a, groups, w, t);
    auto oa = operand_a<O, BM, L::NA>(a, t);
    auto ob = operand_b<O, BN, L::NB>(a, t);
    oa.plan(wave * L::NA, lane, t.ni);
    ob.plan(wave * L::NB, lane, t.nj);
    const Reader<O::ES, O::kACols, BM> ra(lane);
    const ReaderB<O, BN, L::FN> rb(lane);

    // rows split evenly over the two wavefront rows, in 16-row blocks
    const int half = min(BM / 2, (t.ni + 31) / 32 * 16), row0 = uni(wm * half);
    const int nblk = uni(max(0, min(half, t.ni - row0) + 15) / 16);
    ACC acc[L::FM][L::FN];
#pragma unroll
    for (int i = 0; i < L::FM; ++i)
#pragma unroll
        for (int j = 0; j < L::FN; ++j) acc[i][j] = ACC{0, 0, 0, 0};

    const int KT = t.template steps<O>();
    if constexpr (O::ELEM == Elem::f32) {
        if (KT > 0) {
            static_assert(U == 1 && S % 2 == 0, "two sets of operands take turns");
#pragma unroll
            for (int q = 0; q < S; ++q) {
                oa.load(lds + q * L::kStage, wave * L::NA, q);
                ob.load(lds + q * L::kStage + BM * 64, wave * L::NB, q);
            }
            wait_vmcnt<(S - 1) * (L::NA + L::NB)>();
            lds_barrier();
            u32x4_t af[2][L::FM], bf[2][L::FN];
            const int ablk = row0 / 16, bblk = wn * L::FN;
            read_stage<BM>(lds, ablk, bblk, ra, rb, af[0], bf[0]);
            for (int kt = 0; kt < KT;) {
#pragma unroll
                for (int st = 0; st < S; ++st) {              // stages as constants: no addresses to compute
                    if (kt >= KT) break;
                    step_f32<O, BM, BN, S>(lds + (st + 1) % S * L::kStage, lds + st * L::kStage, kt + S, nblk, ablk, bblk, wave,
                                           oa, ob, ra, rb, af[st % 2], bf[st % 2], af[1 - st % 2], bf[1 - st % 2], acc);
                    ++kt;
                }
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
    } else if (KT > 0) {
#pragma unroll
        for (int q = 0; q < (S - 1) * U; ++q) {
            oa.load(lds + q * L::kSub, wave * L::NA, q);
            ob.load(lds + q * L::kSub + BM * 64, wave * L::NB, q);
        }
        for (int kt = 0; kt < KT;) {                          // steps past the end multiply the zeros their loads read
#pragma unroll
            for (int st = 0; st < S; ++st) {                  // stages as constants: no addresses to compute
                if (kt >= KT) break;
                wait_vmcnt<(S - 2) * U * (L::NA + L::NB)>();
                lds_barrier();
                u32x4_t af[U][L::FM], bf[U][L::FN];
                const int nx = (st + S - 1) % S;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    read_and_load<O, BM, BN, 4>(lds + st * L::kStage + u * L::kSub, lds + nx * L::kStage + u * L::kSub,
                                                kt + (S - 1) * U + u, row0 / 16, wn * L::FN, wave, oa, ob, ra, rb, af[u], bf[u]);
                wait_lds();
#pragma unroll
                for (int u = 0; u < U; ++u) mma_step<O::ELEM>(af[u], bf[u], acc, nblk);
                kt += U;
            }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // the last loads (zeros) land before LDS is reused
        __syncthreads();
    }

    const int J = O::KIND == 1 ? a.K : a.N;
    typedef __attribute__((address_space(3))) bf16_t lds_bf16;
    lds_bf16* sC = reinterpret_cast<lds_bf16*>(lds);
    if constexpr (O::kGated) {
        // h, then the projections where they are kept; bf16 through LDS as whole rows
        for (int which = 0; which < (a.ca ? 3 : 1); ++which) {
            if (which) __syncthreads();                       // the tensor before has been read
            OUT* out = (OUT*)(which == 0 ? a.c : which == 1 ? a.ca : a.cb);
#pragma unroll
            for (int i = 0; i < L::FM; ++i) {
                if (i >= nblk) break;
                const int r = row0 + 16 * i + 4 * lq;
#pragma unroll
                for (int j = 0; j < L::FN / 2; ++j) {
                    const int col = wn * (L::kCols / 2) + 16 * j + l16;
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const float p = acc[i][j][v], q = acc[i][L::FN / 2 + j][v];
                        const float val = which == 0 ? gated<O::ELEM>(p, q) : which == 1 ? p : q;
                        if constexpr (sizeof(OUT) == 2) {
                            sC[(r + v) * L::kCS + col] = f32_to_bf16(val);
                        } else {
                            if (r + v < t.ni && col < t.nj) out[(t.crow + r + v) * J + t.j0 + col] = val;
                        }
                    }
                }
            }
            if constexpr (sizeof(OUT) == 2) {
                __syncthreads();
                constexpr int CPR = L::kCols / 8;
                for (int c = tid; c < t.ni * CPR; c += 256) {
                    const int r = c / CPR, cc = (c % CPR) * 8;
                    if (cc < t.nj)
                        __builtin_nontemporal_store(
                            *reinterpret_cast<const __attribute__((address_space(3))) u32x4_t*>(sC + r * L::kCS + cc),
                            reinterpret_cast<u32x4_t*>(out + (t.crow + r) * J + t.j0 + cc));
                }
            }
        }
        return;
    }
    float wsc[L::FN];
    if constexpr (O::ELEM == Elem::i8)
#pragma unroll
        for (int j = 0; j < L::FN; ++j) {
            const int col = wn * (BN / 2) + 16 * j + l16;
            wsc[j] = col < t.nj ? a.ws[(long long)t.e * a.N + t.j0 + col] : 0.f;
        }
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

template <typename O, int BM, int BN, int S, int U, typename OUT>
hipError_t go(const MmArgs& a, hipStream_t st) {
    constexpr size_t lds = Mid<O, BM, BN, S, U>::kLds;
    hipError_t e = allow_lds<k_mm_mid<O, BM, BN, S, U, OUT>>(lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_mm_mid<O, BM, BN, S, U, OUT>), dim3((unsigned)mm_blocks(a, O::KIND, BM, tile_cols<O>(BN)), pair_rows<O>(a)),
                       dim3(256), lds, st, a);
    return hipGetLastError();
}

template <int BM, int BN, int S, int U>
hipError_t go_16(int kind, bool f, const MmArgs& a, hipStream_t st) {
    switch (kind) {
        case 0: return go<Op<0, Elem::bf16>, BM, BN, S, U, bf16_t>(a, st);
        case 1: return go<Op<1, Elem::bf16>, BM, BN, S, U, bf16_t>(a, st);
        case MM_DX_TWO: return go<Op<1, Elem::bf16, Var::two>, BM, BN, S, U, bf16_t>(a, st);
        case 2: return f ? go<Op<2, Elem::bf16>, BM, BN, S, U, float>(a, st) : go<Op<2, Elem::bf16>, BM, BN, S, U, bf16_t>(a, st);
        default: return f ? go<Op<3, Elem::i8>, BM, BN, S, U, float>(a, st) : go<Op<3, Elem::i8>, BM, BN, S, U, bf16_t>(a, st);
    }
}

hipError_t go_32(int kind, const MmArgs& a, hipStream_t st) {
    switch (kind) {
        case 0: return go<Op<0, Elem::f32>, 64, 64, 4, 1, float>(a, st);
        case 1: return go<Op<1, Elem::f32>, 64, 64, 4, 1, float>(a, st);
        case MM_GATED: return go<Op<0, Elem::f32, Var::gated>, 64, 128, 4, 1, float>(a, st);
        case MM_DX_TWO: return go<Op<1, Elem::f32, Var::two>, 64, 64, 4, 1, float>(a, st);
        default: return go<Op<2, Elem::f32>, 64, 64, 4, 1, float>(a, st);
    }
}

}  // namespace

// Two steps a barrier for tiles of 64 (16 and 8 bits): 256 rows, 4096 x 4096 transposed 22.8 ->
// 21.6 us, 512 rows 34.7 -> 32.8, int8 19.0 -> 17.3; tiles of 128 and fp32, whose steps are
// longer, lose by it (208 rows a group, fp32 weight gradient 89 -> 96).  fp32 has tiles of 64 only.
hipError_t launch_mm_mid(int tile, int kind, int dtype, int out_dtype, const MmArgs& a, hipStream_t st) {
    if (kind != 3 && dtype == MOE_F32) return go_32(kind, a, st);
    const bool f = out_dtype == MOE_F32;
    if (kind == MM_GATED)                                     // 64 columns of h either way
        return tile == 64 ? go<Op<0, Elem::bf16, Var::gated>, 64, 128, 4, 1, bf16_t>(a, st)
                          : go<Op<0, Elem::bf16, Var::gated>, 128, 128, 4, 1, bf16_t>(a, st);
    return tile == 64 ? go_16<64, 64, 3, 2>(kind, f, a, st) : go_16<128, 128, 4, 1>(kind, f, a, st);
}

}  // namespace moe
