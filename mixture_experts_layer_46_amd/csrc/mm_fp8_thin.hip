// Grouped products of 8-bit floating-point rows and experts with few rows per group: 16 or 32
// rows by 64 columns, the contraction's blocks of 128 dealt out to the workgroup's wavefronts
// (the mathematics: mm_fp8.h; the form: mm_thin.hip).
//
// What counts is the bytes in flight while the experts stream by.  A wavefront's stage is one
// block: 128 bytes of every index, as two steps of 64, and one more load of the exponents, four
// bytes for each row and for the columns.
#include "mm_fp8.h"

namespace moe {

namespace {

using O = OpF8;
constexpr int kBN = 64;

template <int RB, int W, int S>
struct Thin8 {
    static constexpr int BM = 16 * RB, NA = RB, NB = kBN / 16;
    static constexpr int kSub = (BM + kBN) * 64, kExp = 2 * kSub, kStage = kExp + 256;
    static constexpr int kPer = 2 * (NA + NB) + 1;            // loads of a stage
    static constexpr size_t kRing = (size_t)W * S * kStage, kSums = (size_t)W * BM * kBN * 4;
    static constexpr size_t kLds = kRing > kSums ? kRing : kSums;
};

// Starts the loads of block `kb`.  `exps`: this lane's row of exponents.
template <typename L, typename OA, typename OB>
__device__ __forceinline__ void load_block(lds_char* wr, int kb, int last, const uint8_t* exps, const OA& oa, const OB& ob) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        oa.load(wr + u * L::kSub, 0, 2 * kb + u);
        ob.load(wr + u * L::kSub + L::BM * 64, 0, 2 * kb + u);
    }
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(exps + min(kb >> 2, last) * 4),
                                     (lds_void*)(wr + L::kExp), 4, 0, 0);
}

// Starts a later block's loads into stage `wr`, waits for this block's stage `rd` and reads it
// (separate __restrict__ arguments: see read_and_load in mm_tile.h).
template <typename L, int S, int RB, typename OA, typename OB, typename RA, typename RBt>
__device__ __attribute__((always_inline)) inline void load_and_read(const lds_char* __restrict__ rd, lds_char* __restrict__ wr,
                                                                    int kb, int last, const uint8_t* exps, int lane,
                                                                    const OA& oa, const OB& ob, const RA& ra, const RBt& rb,
                                                                    u32x4_t (&af)[2][RB], u32x4_t (&bf)[2][4],
                                                                    uint32_t (&sx)[RB], uint32_t& sw) {
    load_block<L>(wr, kb, last, exps, oa, ob);
    wait_vmcnt<(S - 1) * L::kPer>();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int i = 0; i < RB; ++i) af[u][i] = ra(rd + u * L::kSub, i);
#pragma unroll
        for (int j = 0; j < 4; ++j) bf[u][j] = rb(rd + u * L::kSub + L::BM * 64, j);
    }
    typedef const __attribute__((address_space(3))) uint32_t lds_cu1;
    lds_cu1* e = (lds_cu1*)(rd + L::kExp);
#pragma unroll
    for (int i = 0; i < RB; ++i) sx[i] = e[16 * i + (lane & 15)];
    sw = e[32];
    __builtin_amdgcn_sched_barrier(0);
    wait_lds();                                               // read: the next block may refill this stage
    __builtin_amdgcn_sched_barrier(0);
}

template <int RB, int W, int S, typename OUT>
__global__ __launch_bounds__(W * 64, 1) void k_mm_fp8_thin(Fp8Args a) {
#ifdef __HIP_DEVICE_COMPILE__          // the host pass needs the signature only
    using L = Thin8<RB, W, S>;
    extern __shared__ uint4 smem[];
    __shared__ Groups groups;
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), l16 = lane & 15, lq = lane >> 4;

    Tile2 t;
    const int w = item_of_block(blockIdx.x, gridDim.x);
    if (w >= count_items<O, L::BM, kBN, OUT>(a.m, groups)) return;
    tile_of_item<O, L::BM, kBN>(a.m, groups, w, t);
    auto oa = operand_a<O, L::BM, L::NA>(a.m, t);
    auto ob = operand_b<O, kBN, L::NB>(a.m, t);
    oa.plan(0, lane, t.ni);
    ob.plan(0, lane, t.nj);
    const Reader<1, false, L::BM> ra(lane);
    const Reader<1, false, kBN> rb(lane);
    // lanes 0..31: the tile's rows; the upper lanes: the columns' block of 128
    const long long sb = fp8_scale_bytes(a.m.K), nb = (a.m.N + 127) / 128;
    const int last = (int)(sb / 4) - 1;
    const uint8_t* exps = lane < 32 ? a.xs + min((long long)t.i0 + min(lane, max(t.ni - 1, 0)), (long long)a.m.rows - 1) * sb
                                    : a.ws + (t.e * nb + t.j0 / 128) * sb;
    f32x4_t acc[RB][4];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    const int KB = (t.C + 127) / 128;
    lds_char* ring = lds + wave * (S * L::kStage);
#pragma unroll
    for (int s = 0; s < S - 1; ++s) load_block<L>(ring + s * L::kStage, wave + s * W, last, exps, oa, ob);
    int st = 0, nx = S - 1;                                   // stage of this block, and of the loads it starts
    for (int kb = wave; kb < KB; kb += W) {
        u32x4_t af[2][RB], bf[2][4];
        uint32_t sx[RB], sw;
        load_and_read<L, S>(ring + st * L::kStage, ring + nx * L::kStage, kb + (S - 1) * W, last, exps, lane, oa, ob, ra, rb, af,
                            bf, sx, sw);
        const int shift = (kb & 3) * 8;
        sw = sw >> shift & 255;
#pragma unroll
        for (int i = 0; i < RB; ++i) sx[i] = sx[i] >> shift & 255;
        if constexpr (sizeof(OUT) == 4) {
            block_f32(af, bf, sx, sw, acc);
        } else {
            auto both = [](u32x4_t lo, u32x4_t hi) {
                return __builtin_bit_cast(i32x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            };
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        both(bf[0][j], bf[1][j]), both(af[0][i], af[1][i]), acc[i][j], 0, 0, 0, (int)sw, 0, (int)sx[i]);
        }
        st = st + 1 == S ? 0 : st + 1;
        nx = nx + 1 == S ? 0 : nx + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");          // the last loads land before LDS is reused
    __syncthreads();

    // sums [wave][row][column], added in wavefront order
    typedef __attribute__((address_space(3))) float lds_float;
    typedef __attribute__((address_space(3))) f32x4_t lds_f4;
    lds_float* sums = reinterpret_cast<lds_float*>(lds);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *(lds_f4*)(sums + (wave * L::BM + 16 * i + l16) * kBN + 16 * j + 4 * lq) = acc[i][j];
    __syncthreads();
    for (int c = tid; c < t.ni * (kBN / 8); c += W * 64) {
        const int r = c / (kBN / 8), cc = (c % (kBN / 8)) * 8;
        if (cc >= t.nj) continue;
        float o[8] = {};
        for (int v = 0; v < W; ++v)
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] += sums[(v * L::BM + r) * kBN + cc + q];
        OUT* p = (OUT*)a.m.c + (t.crow + r) * a.m.N + t.j0 + cc;
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

template <int RB, int W, int S, typename OUT>
hipError_t go(const Fp8Args& a, hipStream_t st) {
    constexpr size_t lds = Thin8<RB, W, S>::kLds;
    const hipError_t e = allow_lds<k_mm_fp8_thin<RB, W, S, OUT>>(lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_mm_fp8_thin<RB, W, S, OUT>), dim3((unsigned)mm_blocks(a.m, 3, 16 * RB, kBN)), dim3(W * 64), lds, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_thin(int rows, int out_dtype, const Fp8Args& a, hipStream_t st) {
    if (rows == 16) return out_dtype == MOE_F32 ? go<1, 4, 3, float>(a, st) : go<1, 4, 3, bf16_t>(a, st);
    return out_dtype == MOE_F32 ? go<2, 4, 3, float>(a, st) : go<2, 4, 3, bf16_t>(a, st);
}

}  // namespace moe
