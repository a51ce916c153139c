// Grouped products with few output tiles: few rows per group (kinds 0, 1 and 3 of mm_tile.h),
// or weight gradients (kind 2) of few small matrices.  16 or 32 rows by 64 columns, the
// contraction split over the workgroup's wavefronts.
//
// Such products stream the matrices once and do little else, so what counts is the bytes in
// flight.  Each of W wavefronts takes every W-th step of the contraction for the whole tile,
// in LDS stages of its own: no barrier and no other wavefront's loads stand between it and
// memory.  At the end the wavefronts' sums meet in LDS and are added in wavefront order (so
// the result does not depend on scheduling), scaled and rounded once.
//
// 8 experts of 2 rows, 4096 x 14336 bf16: 140 us, 5.9 TB/s (16-row tiles 147); one row, 4096 x
// 4096: 10.9 us with 16-row tiles, whose eight wavefronts have twice the steps in flight
// (32-row 11.3, tiles of 64 19).  Three stages: four and six measured the same.  Weight
// gradients of one group, 32-row tiles against tiles of 64: 10314 rows, 80 x 88 bf16 19.0 and
// 43.5 us; 37924 rows, 144 x 120 fp32 340 and 753.
#include "mm_tile.h"

namespace moe {

namespace {

constexpr int kBN = 64;

template <int RB, int W, int S>
struct Thin {
    static constexpr int BM = 16 * RB, NA = RB, NB = kBN / 16;
    static constexpr int kA = BM * 64, kStage = (BM + kBN) * 64;
    static constexpr size_t kRing = (size_t)W * S * kStage, kSums = (size_t)W * BM * kBN * 4;
    static constexpr size_t kLds = kRing > kSums ? kRing : kSums;
};

// Starts the loads of a later step into stage `wr` (read in the previous step), waits for
// this step's stage `rd` and reads it.  The two are separate __restrict__ arguments:
// otherwise the compiler takes the reads to touch what is in flight, and waits for every
// load before them.
template <typename O, int RB, int W, int S, typename OA, typename OB, typename RA, typename RBt>
__device__ __attribute__((always_inline)) inline void load_and_read(const lds_char* __restrict__ rd,
                                                                    lds_char* __restrict__ wr, int kt, const OA& oa,
                                                                    const OB& ob, const RA& ra, const RBt& rb,
                                                                    u32x4_t (&af)[RB], u32x4_t (&bf)[4]) {
    using L = Thin<RB, W, S>;
    oa.load(wr, 0, kt);
    ob.load(wr + L::kA, 0, kt);
    wait_vmcnt<(S - 1) * (L::NA + L::NB)>();
#pragma unroll
    for (int i = 0; i < RB; ++i) af[i] = ra(rd, i);
#pragma unroll
    for (int j = 0; j < 4; ++j) bf[j] = rb(rd + L::kA, j);
    __builtin_amdgcn_sched_barrier(0);
    wait_lds();                                               // read: the next step may refill this stage
    __builtin_amdgcn_sched_barrier(0);
}

template <typename O, int RB, int W, int S, typename OUT>
__global__ __launch_bounds__(W * 64, 2) void k_mm_thin(MmArgs a) {
#ifdef __HIP_DEVICE_COMPILE__          // the host pass needs the signature only
    using L = Thin<RB, W, S>;
    using ACC = typename O::Acc;
    extern __shared__ uint4 smem[];
    __shared__ Groups groups;
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), l16 = lane & 15, lq = lane >> 4;

    Tile2 t;
    const int w = item_of_block(blockIdx.x, gridDim.x);
    if (w >= count_items<O, L::BM, kBN, OUT>(a, groups)) return;
    tile_of_item<O, L::BM, kBN>(a, groups, w, t);
    auto oa = operand_a<O, L::BM, L::NA>(a, t);
    auto ob = operand_b<O, kBN, L::NB>(a, t);
    oa.plan(0, lane, t.ni);
    ob.plan(0, lane, t.nj);
    const Reader<O::ES, O::kACols, L::BM> ra(lane);
    const Reader<O::ES, O::kBCols, kBN> rb(lane);
    ACC acc[RB][4];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = ACC{0, 0, 0, 0};

    const int KT = (t.C + O::kStep - 1) / O::kStep;
    lds_char* ring = lds + wave * (S * L::kStage);
#pragma unroll
    for (int s = 0; s < S - 1; ++s) {
        oa.load(ring + s * L::kStage, 0, wave + s * W);
        ob.load(ring + s * L::kStage + L::kA, 0, wave + s * W);
    }
    int st = 0, nx = S - 1;                                   // stage of this step, and of the loads it starts
    for (int kt = wave; kt < KT; kt += W) {
        u32x4_t af[RB], bf[4];
        load_and_read<O, RB, W, S>(ring + st * L::kStage, ring + nx * L::kStage, kt + (S - 1) * W, oa, ob, ra, rb, af, bf);
        mma_step<O::ELEM>(af, bf, acc, RB);
        st = st + 1 == S ? 0 : st + 1;
        nx = nx + 1 == S ? 0 : nx + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");          // the last loads (zeros) land before LDS is reused
    __syncthreads();

    // sums [wave][row][column], 4 bytes each
    typedef __attribute__((address_space(3))) int lds_int;
    lds_int* sums = reinterpret_cast<lds_int*>(lds);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const auto x = acc[i][j][v];
                int bits;
                if constexpr (O::ELEM == Elem::i8) bits = x;
                else bits = __float_as_int(x);
                sums[(wave * L::BM + 16 * i + 4 * lq + v) * kBN + 16 * j + l16] = bits;
            }
    __syncthreads();
    const int J = O::KIND == 1 ? a.K : a.N;
    // eight consecutive columns of a row per thread
    for (int c = tid; c < t.ni * (kBN / 8); c += W * 64) {
        const int r = c / (kBN / 8), cc = (c % (kBN / 8)) * 8;
        if (cc >= t.nj) continue;
        float o[8];
        if constexpr (O::ELEM == Elem::i8) {
            int s[8] = {};
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int q = 0; q < 8; ++q) s[q] += sums[(w * L::BM + r) * kBN + cc + q];
            const float xs = a.xs[t.i0 + r];
            const float* ws = a.ws + (long long)t.e * a.N + t.j0 + cc;
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = (float)s[q] * xs * ws[q];
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = 0.f;
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int q = 0; q < 8; ++q) o[q] += __int_as_float(sums[(w * L::BM + r) * kBN + cc + q]);
        }
        OUT* p = (OUT*)a.c + (t.crow + r) * J + t.j0 + cc;
        if constexpr (sizeof(OUT) == 2) {
            *reinterpret_cast<uint4*>(p) = uint4{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                                                 pack_bf16x2(o[6], o[7])};
        } else {
            reinterpret_cast<float4*>(p)[0] = make_float4(o[0], o[1], o[2], o[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(o[4], o[5], o[6], o[7]);
        }
    }
#endif
}

template <typename O, int RB, int W, int S, typename OUT>
hipError_t go(const MmArgs& a, hipStream_t st) {
    constexpr size_t lds = Thin<RB, W, S>::kLds;
    hipError_t e = allow_lds<k_mm_thin<O, RB, W, S, OUT>>(lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_mm_thin<O, RB, W, S, OUT>), dim3((unsigned)mm_blocks(a, O::KIND, 16 * RB, kBN)), dim3(W * 64), lds, st, a);
    return hipGetLastError();
}

template <int RB, int W, int S>
hipError_t go_kind(int kind, int dtype, int out_dtype, const MmArgs& a, hipStream_t st) {
    if (kind == 3)
        return out_dtype == MOE_F32 ? go<Op<3, Elem::i8>, RB, W, S, float>(a, st)
                                    : go<Op<3, Elem::i8>, RB, W, S, bf16_t>(a, st);
    if constexpr (RB == 2)
        if (kind == 2) {
            if (dtype == MOE_F32) return go<Op<2, Elem::f32>, RB, W, S, float>(a, st);
            return out_dtype == MOE_F32 ? go<Op<2, Elem::bf16>, RB, W, S, float>(a, st)
                                        : go<Op<2, Elem::bf16>, RB, W, S, bf16_t>(a, st);
        }
    if (dtype == MOE_F32)
        return kind == 0 ? go<Op<0, Elem::f32>, RB, W, S, float>(a, st) : go<Op<1, Elem::f32>, RB, W, S, float>(a, st);
    return kind == 0 ? go<Op<0, Elem::bf16>, RB, W, S, bf16_t>(a, st) : go<Op<1, Elem::bf16>, RB, W, S, bf16_t>(a, st);
}

}  // namespace

// 16 rows: eight wavefronts, for the fewest workgroups; 32 rows: four, and two workgroups a
// CU.  Three stages each.  Measured against 16 rows with four wavefronts and 64 rows with
// four or eight, which no rule on the sizes made pay.
hipError_t launch_mm_thin(int rows, int kind, int dtype, int out_dtype, const MmArgs& a, hipStream_t st) {
    return rows == 16 ? go_kind<1, 8, 3>(kind, dtype, out_dtype, a, st) : go_kind<2, 4, 3>(kind, dtype, out_dtype, a, st);
}

}  // namespace moe
