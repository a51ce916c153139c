// Grouped products of 8-bit floating-point rows and experts, tiles of 256, 128 and 64 (the
// mathematics and the operands: mm_fp8.h).
//
// Both kernels are shaped as those of the other grouped products: 256 x 256 tiles by two groups
// of four wavefronts half a step apart (mm.hip), and smaller tiles by four wavefronts with
// several workgroups a CU (mm_mid.hip).
#include "mm_fp8.h"
#include "mm_large.h"

namespace moe {

namespace {

using namespace large;
using O = OpF8;
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) u32x2_t lds_u2;
typedef const __attribute__((address_space(3))) u32x4_t lds_cu4;

using OpA8 = Operand<1, false, kT, kLoads, true>;

constexpr int kCS = kT + 8;                   // bf16 per row of the output staging tile
constexpr size_t kLds = (size_t)kT * kCS * 2; // staging tile; the stages (128 KB) and the exponents' slots lie inside
static_assert(kStages * kStage + ExpLoads<8>::kBytes <= (int)kLds, "stages and exponents fit below the staging tile's end");

// The 32 x 32 block `c`: lane l holds row l & 31 and columns 8 q + 4 (l >> 5) .. + 3, q = 0 .. 3.
__device__ __forceinline__ void put_block(const f32x16_t& c, lds_char* stage, int cs, int r, int col) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        *(lds_u2*)(stage + (r * cs + col + 8 * q) * 2) =
            u32x2_t{pack_bf16x2(c[4 * q], c[4 * q + 1]), pack_bf16x2(c[4 * q + 2], c[4 * q + 3])};
}
template <int BN, int NT>
__device__ __forceinline__ void put_rows(const lds_char* stage, int cs, const MmArgs& a, const Tile2& t, int tid) {
    constexpr int CPR = BN / 8;
    for (int c = tid; c < t.ni * CPR; c += NT) {
        const int r = c / CPR, cc = (c % CPR) * 8;
        if (cc < t.nj)
            __builtin_nontemporal_store(*(lds_cu4*)(stage + (r * cs + cc) * 2),
                                        reinterpret_cast<u32x4_t*>((bf16_t*)a.c + (t.crow + r) * a.N + t.j0 + cc));
    }
}

// Reads a wavefront's operands of a step from stage `rd` and starts its share of a later step's
// loads into stage `wr` (separate __restrict__ arguments: see read_and_load in mm_tile.h).
template <int TA, int TB, int W, int FM, int FN, typename OA, typename OB>
__device__ __attribute__((always_inline)) inline void read_and_load8(const lds_char* __restrict__ rd,
                                                                     lds_char* __restrict__ wr, int kt, int ablk, int bblk,
                                                                     int wave, const OA& oa, const OB& ob,
                                                                     const Reader32& rr, i32x8_t (&af)[FM],
                                                                     i32x8_t (&bf)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i) af[i] = rr(rd, ablk + i);
#pragma unroll
    for (int j = 0; j < FN; ++j) bf[j] = rr(rd + TA * 64, bblk + j);
    __builtin_amdgcn_sched_barrier(0);
    oa.load(wr, wave * (TA / 16 / W), kt);
    ob.load(wr + TA * 64, wave * (TB / 16 / W), kt);
}

__device__ __forceinline__ void wait_stage(int kt) {
    if (((kt - 4) & 7) < 2) wait_vmcnt<kVmcnt + 1>();
    else wait_vmcnt<kVmcnt>();
}

// The steps of one of the two wavefront groups; barriers and waits as in mm.hip.  An exponents'
// load goes out between the stage loads of steps kt - 1 and kt = 4 (mod 8): there and one step
// later it may be in flight too when the stage of step kt + 1 is waited for.
template <int GROUP>
__device__ __attribute__((always_inline)) inline void steps(lds_char* lds, int KT, int nblk, int ablk, int wn, int wave,
                                                            const OpA8& oa, const OpA8& ob, const Reader32& rr,
                                                            const ExpLoads<8>& el, int lane, f32x16_t (&acc)[4][2]) {
    i32x8_t af[4], bf[2];
    Exps<4> ex;
    lds_char* slots = lds + kStages * kStage;
    if constexpr (GROUP == 1) lds_barrier();
    for (int kt = 0; kt < KT; ++kt) {
        ex.step(el, slots, kt, ablk, wn >> 1, lane);
        if ((kt & 7) == 4) el.load(slots, wave, kt + 4);
        read_and_load8<kT, kT, 8>(lds + (kt % kStages) * kStage, lds + ((kt + 3) % kStages) * kStage, kt + 3, ablk, wn * 2,
                                  wave, oa, ob, rr, af, bf);
        wait_lds();
        if constexpr (GROUP == 1) wait_stage(kt);
        lds_barrier();
        asm volatile("" : "+s"(nblk));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (__builtin_expect(i < nblk, 1)) {
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = mma32(bf[j], af[i], acc[i][j], ex.w, ex.x[i]);
            }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) asm volatile("" : "+a"(acc[i][j]));
        if constexpr (GROUP == 0) wait_stage(kt);
        lds_barrier();
    }
    if constexpr (GROUP == 0) lds_barrier();
}

__global__ __launch_bounds__(512, 1) void k_mm_fp8(Fp8Args a) {
#ifdef __HIP_DEVICE_COMPILE__          // the host pass needs the signature only
    extern __shared__ uint4 smem[];
    __shared__ Groups groups;
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), wm = wave >> 2, wn = wave & 3;

    const int w = item_of_block(blockIdx.x, gridDim.x);
    if (w >= count_items<O, kT, kT, bf16_t>(a.m, groups)) return;
    Tile2 t;
    tile_of_item<O, kT, kT>(a.m, groups, w, t);
    auto oa = operand_a<O, kT, kLoads, true>(a.m, t);
    auto ob = operand_b<O, kT, kLoads, true>(a.m, t);
    oa.plan(wave * kLoads, lane, t.ni);
    ob.plan(wave * kLoads, lane, t.nj);

    // this wavefront's rows, in 32-row blocks: the tile's, split evenly over the two groups
    const int half = min(128, (t.ni + 63) / 64 * 32), row0 = uni(wm * half);
    const int nblk = uni(max(0, min(half, t.ni - row0) + 31) / 32);
    f32x16_t acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x16_t{};

    const int KT = (t.C + 63) / 64;
    {
        const Reader32 rr(lane);
        ExpLoads<8> el;
        el.plan(a, t, wave, lane);
        el.load(lds + kStages * kStage, wave, 0);
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            oa.load(lds + s * kStage, wave * kLoads, s);
            ob.load(lds + s * kStage + kT * 64, wave * kLoads, s);
        }
        wait_vmcnt<kVmcnt>();
        lds_barrier();
        if (wm == 0) steps<0>(lds, KT, nblk, row0 / 32, wn, wave, oa, ob, rr, el, lane, acc);
        else steps<1>(lds, KT, nblk, row0 / 32, wn, wave, oa, ob, rr, el, lane, acc);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // the last loads (zeros) land before LDS is reused
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= nblk) break;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            put_block(acc[i][j], lds, kCS, row0 + 32 * i + (lane & 31), wn * 64 + 32 * j + 4 * (lane >> 5));
    }
    __syncthreads();
    put_rows<kT, 512>(lds, kCS, a.m, t, tid);
#endif
}

// Tiles of B x B, U steps a barrier, S stages.
template <int B, int S, int U>
struct Mid8 {
    static constexpr int F = B / 64, NL = B / 64;             // 32-index blocks of a wavefront; loads per operand and step
    static constexpr int kSub = 2 * B * 64, kStage = U * kSub, kCS = B + 8;
    static constexpr size_t kOut = (size_t)B * kCS * 2;
    static constexpr size_t kIn = (size_t)S * kStage + ExpLoads<4>::kBytes, kLds = kOut > kIn ? kOut : kIn;
};

template <int B, int S, int U>
__global__ __launch_bounds__(256, 2) void k_mm_fp8_mid(Fp8Args a) {
#ifdef __HIP_DEVICE_COMPILE__          // the host pass needs the signature only
    using L = Mid8<B, S, U>;
    extern __shared__ uint4 smem[];
    __shared__ Groups groups;
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), wm = wave >> 1, wn = wave & 1;

    const int w = item_of_block(blockIdx.x, gridDim.x);
    if (w >= count_items<O, B, B, bf16_t>(a.m, groups)) return;
    Tile2 t;
    tile_of_item<O, B, B>(a.m, groups, w, t);
    auto oa = operand_a<O, B, L::NL, true>(a.m, t);
    auto ob = operand_b<O, B, L::NL, true>(a.m, t);
    oa.plan(wave * L::NL, lane, t.ni);
    ob.plan(wave * L::NL, lane, t.nj);
    const Reader32 rr(lane);

    const int half = min(B / 2, (t.ni + 63) / 64 * 32), row0 = uni(wm * half);
    const int nblk = uni(max(0, min(half, t.ni - row0) + 31) / 32);
    f32x16_t acc[L::F][L::F];
#pragma unroll
    for (int i = 0; i < L::F; ++i)
#pragma unroll
        for (int j = 0; j < L::F; ++j) acc[i][j] = f32x16_t{};

    const int KT = (t.C + 63) / 64;
    ExpLoads<4> el;
    Exps<L::F> ex;
    lds_char* slots = lds + S * L::kStage;
    el.plan(a, t, wave, lane);
    el.load(slots, wave, 0);
#pragma unroll
    for (int q = 0; q < (S - 1) * U; ++q) {
        oa.load(lds + q * L::kSub, wave * L::NL, q);
        ob.load(lds + q * L::kSub + B * 64, wave * L::NL, q);
    }
    for (int kt = 0; kt < KT;) {                              // a step past the end multiplies the zeros its loads read
#pragma unroll
        for (int st = 0; st < S; ++st) {                      // stages as constants: no addresses to compute
            if (kt >= KT) break;
            wait_vmcnt<(S - 2) * U * 2 * L::NL>();
            lds_barrier();
            if ((kt & 7) == 4) el.load(slots, wave, kt + 4);
            i32x8_t af[U][L::F], bf[U][L::F];
            const int nx = (st + S - 1) % S;
#pragma unroll
            for (int u = 0; u < U; ++u)
                read_and_load8<B, B, 4>(lds + st * L::kStage + u * L::kSub, lds + nx * L::kStage + u * L::kSub,
                                        kt + (S - 1) * U + u, row0 / 32, wn * L::F, wave, oa, ob, rr, af[u], bf[u]);
            ex.step(el, slots, kt, row0 / 32, 0, lane);
            wait_lds();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                int rows = nblk;
                if constexpr (L::F > 1) asm volatile("" : "+s"(rows));
#pragma unroll
                for (int i = 0; i < L::F; ++i)
                    if (__builtin_expect(i < rows, 1)) {
#pragma unroll
                        for (int j = 0; j < L::F; ++j) acc[i][j] = mma32(bf[u][j], af[u][i], acc[i][j], ex.w, ex.x[i]);
                    }
            }
            kt += U;
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");          // the last loads (zeros) land before LDS is reused
    __syncthreads();
#pragma unroll
    for (int i = 0; i < L::F; ++i) {
        if (i >= nblk) break;
#pragma unroll
        for (int j = 0; j < L::F; ++j)
            put_block(acc[i][j], lds, L::kCS, row0 + 32 * i + (lane & 31), wn * (B / 2) + 32 * j + 4 * (lane >> 5));
    }
    __syncthreads();
    put_rows<B, 256>(lds, L::kCS, a.m, t, tid);
#endif
}

// fp32 output: tiles of 64 x 64, a block of 128 (two steps) a stage, with exact operands.
struct Exact8 {
    static constexpr int B = 64, S = 3, kSub = 2 * B * 64, kStage = 2 * kSub;
    static constexpr size_t kLds = (size_t)S * kStage + ExpLoads<4>::kBytes;
};

__device__ __attribute__((always_inline)) inline void read_and_load_exact(const lds_char* __restrict__ rd,
                                                                          lds_char* __restrict__ wr, int kt, int ablk, int bblk,
                                                                          int wave, const Operand<1, false, 64, 1>& oa,
                                                                          const Operand<1, false, 64, 1>& ob,
                                                                          const Reader<1, false, 64>& rr, u32x4_t (&af)[2],
                                                                          u32x4_t (&bf)[2]) {
    read_stage<64>(rd, ablk, bblk, rr, rr, af, bf);
    __builtin_amdgcn_sched_barrier(0);
    oa.load(wr, wave, kt);
    ob.load(wr + 64 * 64, wave, kt);
}

__global__ __launch_bounds__(256, 2) void k_mm_fp8_exact(Fp8Args a) {
#ifdef __HIP_DEVICE_COMPILE__          // the host pass needs the signature only
    using L = Exact8;
    constexpr int B = L::B, S = L::S;
    extern __shared__ uint4 smem[];
    __shared__ Groups groups;
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), wm = wave >> 1, wn = wave & 1;

    const int w = item_of_block(blockIdx.x, gridDim.x);
    if (w >= count_items<O, B, B, float>(a.m, groups)) return;
    Tile2 t;
    tile_of_item<O, B, B>(a.m, groups, w, t);
    auto oa = operand_a<O, B, 1>(a.m, t);
    auto ob = operand_b<O, B, 1>(a.m, t);
    oa.plan(wave, lane, t.ni);
    ob.plan(wave, lane, t.nj);
    const Reader<1, false, B> rr(lane);
    f32x4_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    const int KT = (t.C + 63) / 64;
    ExpLoads<4> el;
    lds_char* slots = lds + S * L::kStage;
    el.plan(a, t, wave, lane);
    el.load(slots, wave, 0);
#pragma unroll
    for (int q = 0; q < (S - 1) * 2; ++q) {
        oa.load(lds + q * L::kSub, wave, q);
        ob.load(lds + q * L::kSub + B * 64, wave, q);
    }
    uint32_t ex[2] = {}, ew = 0;
    for (int kt = 0; kt < KT;) {
#pragma unroll
        for (int st = 0; st < S; ++st) {
            if (kt >= KT) break;
            wait_vmcnt<(S - 2) * 2 * 2>();
            lds_barrier();
            if ((kt & 7) == 4) el.load(slots, wave, kt + 4);
            u32x4_t af[2][2], bf[2][2];
            const int nx = (st + S - 1) % S;
#pragma unroll
            for (int u = 0; u < 2; ++u)
                read_and_load_exact(lds + st * L::kStage + u * L::kSub, lds + nx * L::kStage + u * L::kSub, kt + (S - 1) * 2 + u,
                                    wm * 2, wn * 2, wave, oa, ob, rr, af[u], bf[u]);
            if ((kt & 7) == 0) {
                typedef const __attribute__((address_space(3))) uint32_t lds_cu1;
                lds_cu1* s = (lds_cu1*)(slots + ((kt >> 3) & 1) * ExpLoads<4>::kSlot);
                ex[0] = s[wm * 64 + (lane & 15)];
                ex[1] = s[wm * 64 + 16 + (lane & 15)];
                ew = s[32];
            }
            wait_lds();
            const int shift = (kt & 6) * 4;
            const uint32_t sx[2] = {ex[0] >> shift & 255, ex[1] >> shift & 255};
            block_f32(af, bf, sx, ew >> shift & 255, acc);
            kt += 2;
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");          // no load is left on its way to LDS
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = wm * 32 + 16 * i + (lane & 15), col = wn * 32 + 16 * j + 4 * (lane >> 4);
            if (r < t.ni && col < t.nj) *reinterpret_cast<f32x4_t*>((float*)a.m.c + (t.crow + r) * a.m.N + t.j0 + col) = acc[i][j];
        }
#endif
}

template <auto KERN, int B>
hipError_t go(const Fp8Args& a, int threads, size_t lds, hipStream_t st) {
    const hipError_t e = allow_lds<KERN>(lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(KERN, dim3((unsigned)mm_blocks(a.m, 3, B, B)), dim3(threads), lds, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_large(const Fp8Args& a, hipStream_t st) { return go<k_mm_fp8, kT>(a, 512, kLds, st); }

hipError_t launch_fp8_mid(int tile, const Fp8Args& a, hipStream_t st) {
    return tile == 64 ? go<k_mm_fp8_mid<64, 3, 2>, 64>(a, 256, Mid8<64, 3, 2>::kLds, st)
                      : go<k_mm_fp8_mid<128, 4, 1>, 128>(a, 256, Mid8<128, 4, 1>::kLds, st);
}

hipError_t launch_fp8_exact(const Fp8Args& a, hipStream_t st) { return go<k_mm_fp8_exact, 64>(a, 256, Exact8::kLds, st); }

}  // namespace moe
