// Grouped products of 8-bit floating-point rows and experts with few rows per group: 32 rows (fp32
// output: or 16) by 64 columns, the steps of the contraction dealt out to the workgroup's wavefronts (the
// mathematics: mm_fp8.h; the form: mm_thin.hip).
//
// What counts is the bytes in flight while the experts stream by, and that another workgroup's
// fill the memory's time while one starts or ends.  A stage is one step: 64 bytes of every
// index and one more load of the exponents, four bytes for each row and for the columns.
// 64 experts of 2 rows each, 4096 x 14336: 606 us, 6.2 TB/s, what pure reading reaches; with the 128
// rows drawn at random, so that 53 to 57 of the experts have any, 510 to 545 us at the same rate.
// One row of 4096 x 14336 14 us (4.2 TB/s): its 224 tiles do not fill 256 CUs that hold two
// workgroups each.  (Stages of a whole block for the 16x16x128 instruction leave room for one
// workgroup a CU: 621 to 653 us on the drawn groups.)
#include "mm_fp8.h"

namespace moe {

namespace {

using O = OpF8;
constexpr int kBN = 64;

template <int BM_, int W, int S>
struct Thin8 {
    static constexpr int BM = BM_, NA = BM / 16, NB = kBN / 16;
    static constexpr int kExp = (BM + kBN) * 64, kStage = kExp + 256;
    static constexpr int kPer = NA + NB + 1;                  // loads of a stage
    static constexpr size_t kRing = (size_t)W * S * kStage, kSums = (size_t)W * BM * kBN * 4;
    static constexpr size_t kLds = kRing > kSums ? kRing : kSums;
};

// Starts the loads of step kt.  `exps`: this lane's row of exponents.
template <typename L, typename OA, typename OB>
__device__ __forceinline__ void load_step(lds_char* wr, int kt, int last, const uint8_t* exps, const OA& oa, const OB& ob) {
    oa.load(wr, 0, kt);
    ob.load(wr + L::BM * 64, 0, kt);
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(exps + min(kt >> 3, last) * 4),
                                     (lds_void*)(wr + L::kExp), 4, 0, 0);
}

// Starts a later step's loads into stage `wr`, waits for this step's stage `rd` and reads it with
// `read` (separate __restrict__ arguments: see read_and_load in mm_tile.h).
template <typename L, int S, typename OA, typename OB, typename F>
__device__ __attribute__((always_inline)) inline void load_and_read(const lds_char* __restrict__ rd, lds_char* __restrict__ wr,
                                                                    int kt, int last, const uint8_t* exps, const OA& oa,
                                                                    const OB& ob, const F& read) {
    load_step<L>(wr, kt, last, exps, oa, ob);
    wait_vmcnt<(S - 1) * L::kPer>();
    read(rd, (const __attribute__((address_space(3))) uint32_t*)(rd + L::kExp));
    __builtin_amdgcn_sched_barrier(0);
    wait_lds();                                               // read: the next step may refill this stage
    __builtin_amdgcn_sched_barrier(0);
}

template <int BM, int W, int S, typename OUT>
__global__ __launch_bounds__(W * 64, 2) void k_mm_fp8_thin(Fp8Args a) {
#ifdef __HIP_DEVICE_COMPILE__          // the host pass needs the signature only
    using L = Thin8<BM, W, S>;
    constexpr bool kExact = sizeof(OUT) == 4;                 // bf16 operands, 16 x 16 blocks
    typedef const __attribute__((address_space(3))) uint32_t lds_cu1;
    extern __shared__ uint4 smem[];
    __shared__ Groups groups;
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), l16 = lane & 15, lq = lane >> 4;

    Tile2 t;
    const int w = item_of_block(blockIdx.x, gridDim.x);
    if (w >= count_items<O, BM, kBN, OUT>(a.m, groups)) return;
    tile_of_item<O, BM, kBN>(a.m, groups, w, t);
    auto oa = operand_a<O, BM, L::NA, !kExact>(a.m, t);
    auto ob = operand_b<O, kBN, L::NB, !kExact>(a.m, t);
    oa.plan(0, lane, t.ni);
    ob.plan(0, lane, t.nj);
    // lanes 0..31: the tile's rows; the upper lanes: the columns' block of 128
    const long long sb = fp8_scale_bytes(a.m.K), nb = (a.m.N + 127) / 128;
    const int last = (int)(sb / 4) - 1;
    const uint8_t* exps = lane < 32 ? a.xs + min((long long)t.i0 + min(lane, max(t.ni - 1, 0)), (long long)a.m.rows - 1) * sb
                                    : a.ws + (t.e * nb + t.j0 / 128) * sb;

    const int KT = (t.C + 63) / 64;
    lds_char* ring = lds + wave * (S * L::kStage);
#pragma unroll
    for (int s = 0; s < S - 1; ++s) load_step<L>(ring + s * L::kStage, wave + s * W, last, exps, oa, ob);
    int st = 0, nx = S - 1;                                   // stage of this step, and of the loads it starts
    // sums [wave][row][column], added in wavefront order
    typedef __attribute__((address_space(3))) float lds_float;
    typedef __attribute__((address_space(3))) f32x4_t lds_f4;
    lds_float* sums = reinterpret_cast<lds_float*>(lds);
    if constexpr (kExact) {
        const Reader<1, false, BM> ra(lane);
        const Reader<1, false, kBN> rb(lane);
        f32x4_t acc[L::NA][4];
#pragma unroll
        for (int i = 0; i < L::NA; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        for (int kt = wave; kt < KT; kt += W) {
            u32x4_t af[1][L::NA], bf[1][4];
            uint32_t sx[L::NA], sw;
            const int shift = (kt & 6) * 4;
            load_and_read<L, S>(ring + st * L::kStage, ring + nx * L::kStage, kt + (S - 1) * W, last, exps, oa, ob,
                                [&](const lds_char* rd, lds_cu1* e) {
                                    read_stage<BM>(rd, 0, 0, ra, rb, af[0], bf[0]);
#pragma unroll
                                    for (int i = 0; i < L::NA; ++i) sx[i] = e[16 * i + l16];
                                    sw = e[32];
                                });
#pragma unroll
            for (int i = 0; i < L::NA; ++i) sx[i] = sx[i] >> shift & 255;
            block_f32(af, bf, sx, sw >> shift & 255, L::NA, acc);
            st = st + 1 == S ? 0 : st + 1;
            nx = nx + 1 == S ? 0 : nx + 1;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // the last loads land before LDS is reused
        __syncthreads();
#pragma unroll
        for (int i = 0; i < L::NA; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) *(lds_f4*)(sums + (wave * BM + 16 * i + l16) * kBN + 16 * j + 4 * lq) = acc[i][j];
    } else {
        static_assert(BM == 32, "the instruction's rows");
        const Reader32 rr(lane);
        f32x16_t acc[2] = {};
        for (int kt = wave; kt < KT; kt += W) {
            i32x8_t af, bf[2];
            uint32_t sx, sw;
            load_and_read<L, S>(ring + st * L::kStage, ring + nx * L::kStage, kt + (S - 1) * W, last, exps, oa, ob,
                                [&](const lds_char* rd, lds_cu1* e) {
                                    af = rr(rd, 0);
                                    bf[0] = rr(rd + BM * 64, 0);
                                    bf[1] = rr(rd + BM * 64, 1);
                                    sx = e[lane & 31];
                                    sw = e[32];
                                });
            const int shift = (kt & 6) * 4;
            sx >>= shift;
            sw >>= shift;
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[j] = mma32(bf[j], af, acc[j], sw, sx);
            st = st + 1 == S ? 0 : st + 1;
            nx = nx + 1 == S ? 0 : nx + 1;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // the last loads land before LDS is reused
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(lds_f4*)(sums + (wave * BM + (lane & 31)) * kBN + 32 * j + 8 * q + 4 * (lane >> 5)) =
                    f32x4_t{acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
    }
    __syncthreads();
    for (int c = tid; c < t.ni * (kBN / 8); c += W * 64) {
        const int r = c / (kBN / 8), cc = (c % (kBN / 8)) * 8;
        if (cc >= t.nj) continue;
        float o[8] = {};
        for (int v = 0; v < W; ++v)
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] += sums[(v * BM + r) * kBN + cc + q];
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

template <int BM, int W, int S, typename OUT>
hipError_t go(const Fp8Args& a, hipStream_t st) {
    constexpr size_t lds = Thin8<BM, W, S>::kLds;
    const hipError_t e = allow_lds<k_mm_fp8_thin<BM, W, S, OUT>>(lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_mm_fp8_thin<BM, W, S, OUT>), dim3((unsigned)mm_blocks(a.m, 3, BM, kBN)), dim3(W * 64), lds, st, a);
    return hipGetLastError();
}

}  // namespace

// 16 rows (fp32 output): eight wavefronts, for the fewest workgroups; 32 rows: four, and two
// workgroups a CU.
hipError_t launch_fp8_thin(int rows, int out_dtype, const Fp8Args& a, hipStream_t st) {
    if (rows == 16) return go<16, 8, 3, float>(a, st);
    return out_dtype == MOE_F32 ? go<32, 4, 3, float>(a, st) : go<32, 4, 3, bf16_t>(a, st);
}

}  // namespace moe
