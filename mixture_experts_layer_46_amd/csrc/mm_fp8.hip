// Grouped products of 8-bit floating-point rows and experts, tiles of 256, 128 and 64 (the
// mathematics and the operands: mm_fp8.h).
//
// The kernels are shaped as those of the other grouped products: 256 x 256 tiles by two groups
// of four wavefronts half a step apart (mm.hip), and smaller tiles by four wavefronts with
// several workgroups a CU (mm_mid.hip).  Of the smaller ones, 1 expert of 512 rows of 4096 x 4096
// takes 19 us (917 TFLOP/s), 64 experts of 256 rows of 2048 x 1408 68 us (1390).
//
// The large tiles run at 2600 TFLOP/s on 8192^3, where the card's library reaches 2890 with one
// scale per tensor and a loop of nothing but this instruction 3900: matrix units are busy two
// thirds of the time at a clock that the card's power limit holds at 1.6 to 1.8 of 2.4 GHz:
// schedules of 765, 797 and 814 thousand cycles (loads in the matrix phase, column operands read
// one phase early) all took 440 us.  Four wavefronts of 128 x 128, which read a third
// less from LDS, were slower by 6 to 9%: with one wavefront per SIMD the loads' issue shows.
#include "mm_fp8.h"
#include "mm_large.h"

namespace moe {

namespace {

using namespace large;
using O = OpF8;
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) u32x2_t lds_u2;
typedef const __attribute__((address_space(3))) u32x4_t lds_cu4;

// An operand of the large tiles, two steps at a time: lines of 128 bytes of memory, eight rows to a
// load, so that L2 is asked for whole lines.  Steps of 64 bytes ask for each line twice, which
// a card at its power limit pays for: 8192^3 448 -> 420 us, 8 experts, 8192 rows, 4096 x 14336 498 ->
// 479, with half the requests.  (bf16 tiles in this way were 10% slower.)  In LDS an index keeps
// its 128 bytes as eight 16-byte chunks, chunk q of index m at q ^ ((m >> 1) & 7): the 16 lanes that
// one cycle of a ds_read_b128 serves (see swa4) have eight even and eight odd indexes, whose m / 2
// differ modulo 8.
struct Wide {
    static constexpr int kLoads = 4, kBytes = kT * 128;       // loads per wavefront; bytes of a stage
    uint64_t base;
    uint32_t ld, n, cbytes;
    uint32_t off[kLoads], kq;     // kq: this lane's byte within the two steps, of its even loads
    __device__ __forceinline__ void plan(uint64_t base_, int C, int valid, int wave, int lane) {
        base = base_;
        ld = cbytes = (uint32_t)C;
        n = (uint32_t)valid;
        kq = (uint32_t)((lane & 7) ^ (lane >> 4)) * 16;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = (wave * kLoads + i) * 8 + (lane >> 3);
            off[i] = r < valid ? (uint32_t)r * ld + (kq ^ (i & 1) * 64) : kOOB;
        }
    }
    // loads i0 .. i0 + NL - 1 of double step d
    template <int NL>
    __device__ __forceinline__ void load(lds_char* stage, int wave, int d, int i0) const {
        const uint32_t k0 = min((uint32_t)d * 128, cbytes), left = cbytes - k0;
        const __amdgpu_buffer_rsrc_t r = make_rsrc((const void*)base, n * ld);
#pragma unroll
        for (int i = i0; i < i0 + NL; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(stage + (wave * kLoads + i) * 1024), 16,
                                                     (kq ^ (i & 1) * 64) < left ? off[i] : kOOB, (int)k0, 0, 0);
    }
};
// 32-index block `blk` of step `s` (0, 1) of a stage as a matrix operand (see Reader32).
struct WideReader {
    int rd;
    __device__ __forceinline__ explicit WideReader(int lane) {
        const int m = lane & 31;
        rd = m * 128 + (((lane >> 5) * 2 ^ ((m >> 1) & 7)) << 4);
    }
    __device__ __forceinline__ i32x8_t operator()(const lds_char* stage, int blk, int s) const {
        typedef const __attribute__((address_space(3))) i32x4_t lds_i4;
        const int at = rd ^ s * 64;
        const i32x4_t lo = *(lds_i4*)(stage + blk * 4096 + at), hi = *(lds_i4*)(stage + blk * 4096 + (at ^ 16));
        return i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
};
constexpr int kPair = 2 * Wide::kBytes;       // bytes of a double step: the A operand, then the B operand

constexpr int kCS = kT + 8;                   // bf16 per row of the output staging tile
constexpr size_t kLds = (size_t)kT * kCS * 2; // staging tile; the stages (128 KB) and the exponents' slots lie inside
static_assert(2 * kPair + ExpLoads<8>::kBytes <= (int)kLds, "stages and exponents fit below the staging tile's end");

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

// The steps of one of the two wavefront groups.  Between two barriers one group is in its read
// phase (R) and the other in its matrix phase (M):
//   group 0:  R0 | M0 | R1 | M1 | ... | M(KT-1) | (idle)
//   group 1: (idle) | R0 | M0 | R1 | ... | R(KT-1) | M(KT-1)
// Loads are of double steps, into two stages that take turns, between the matrix instructions: the
// stage of the steps 2d - 2 and 2d - 1 has been read when group 1 enters M(2d-1); there it starts its
// loads of double step d + 1, and group 0 in M(2d).  They are waited for before the barrier that
// opens group 0's R(2d+2), by group 0 at the end of M(2d+1), by group 1 at the end of R(2d+1).
// Exponents are loaded in M(k), k = 4 (mod 8), and read in R(k), k = 0 (mod 8).
__device__ __attribute__((always_inline)) inline void phase_r(const lds_char* __restrict__ rd, int s, int ablk, int bblk,
                                                              const WideReader& rr, i32x8_t (&af)[4], i32x8_t (&bf)[2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) af[i] = rr(rd, ablk + i, s);
#pragma unroll
    for (int j = 0; j < 2; ++j) bf[j] = rr(rd + Wide::kBytes, bblk + j, s);
    wait_lds();
}
// `wr`: the stage that loads of double step d go into (LOADS)
template <bool LOADS>
__device__ __attribute__((always_inline)) inline void phase_m(lds_char* __restrict__ wr, int d, int nblk, int wave, const Wide& oa,
                                                              const Wide& ob, const Exps<4>& ex, const i32x8_t (&af)[4],
                                                              const i32x8_t (&bf)[2], f32x16_t (&acc)[4][2]) {
    asm volatile("" : "+s"(nblk));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (__builtin_expect(i < nblk, 1)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mma32(bf[j], af[i], acc[i][j], ex.w, ex.x[i]);
        }
        if constexpr (LOADS) {
            if (i < 2) oa.load<2>(wr, wave, d, 2 * i);
            else ob.load<2>(wr + Wide::kBytes, wave, d, 2 * i - 4);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) asm volatile("" : "+a"(acc[i][j]));
}

template <int GROUP>
__device__ __attribute__((always_inline)) inline void steps(lds_char* lds, int KT, int nblk, int ablk, int wn, int wave,
                                                            const Wide& oa, const Wide& ob, const WideReader& rr,
                                                            const ExpLoads<8>& el, int lane, f32x16_t (&acc)[4][2]) {
    i32x8_t af[4], bf[2];
    Exps<4> ex;
    lds_char* slots = lds + 2 * kPair;
    if constexpr (GROUP == 1) lds_barrier();
    for (int k0 = 0; k0 < KT; k0 += 4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {                         // stages as constants: no addresses to compute
            const int kt = k0 + q;
            if (kt >= KT) break;
            ex.step(el, slots, kt, ablk, wn >> 1, lane);
            phase_r(lds + q / 2 * kPair, q % 2, ablk, wn * 2, rr, af, bf);
            if constexpr (GROUP == 1)
                if (q % 2 == 1) wait_vmcnt<0>();
            lds_barrier();
            if (q == 0 && (kt & 7) == 4) el.load(slots, wave, kt + 4);
            if constexpr (GROUP == 0) {
                if (q == 0 && kt == 0) phase_m<false>(lds, 0, nblk, wave, oa, ob, ex, af, bf, acc);      // double step 1 is on its way
                else if (q % 2 == 0) phase_m<true>(lds + (q / 2 + 1) % 2 * kPair, kt / 2 + 1, nblk, wave, oa, ob, ex, af, bf, acc);
                else phase_m<false>(lds, 0, nblk, wave, oa, ob, ex, af, bf, acc);
                if (q % 2 == 1) wait_vmcnt<0>();
            } else {
                if (q % 2 == 1) phase_m<true>(lds + q / 2 * kPair, kt / 2 + 2, nblk, wave, oa, ob, ex, af, bf, acc);
                else phase_m<false>(lds, 0, nblk, wave, oa, ob, ex, af, bf, acc);
            }
            lds_barrier();
        }
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
    Wide oa, ob;
    oa.plan(t.abase, t.C, t.ni, wave, lane);
    ob.plan(t.bbase, t.C, t.nj, wave, lane);

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
        const WideReader rr(lane);
        ExpLoads<8> el;
        el.plan(a, t, wave, lane);
        el.load(lds + 2 * kPair, wave, 0);
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            oa.load<4>(lds + d * kPair, wave, d, 0);
            ob.load<4>(lds + d * kPair + Wide::kBytes, wave, d, 0);
        }
        wait_vmcnt<2 * Wide::kLoads>();                       // double step 0
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

// fp32 output: tiles of B x B, a block of 128 (two steps) a stage, with exact operands (mm_fp8.h).
// Opening an operand (8 conversions for 16 indexes and 64 contraction bytes) and adding a block's
// scaled sums are vector instructions beside the matrix ones, and bound it: the wider a
// wavefront's share, the fewer.  8192^3: 64 1423 us (773 TFLOP/s), 128 986 (1115), in which a
// wavefront opens 8 operands for 32 matrix instructions, not 4 for 8.
template <int B, int S>
struct Exact8 {
    static constexpr int F = B / 32, NL = B / 64;             // 16-index blocks of a wavefront; loads per operand and step
    static constexpr int kSub = 2 * B * 64, kStage = 2 * kSub;
    static constexpr size_t kLds = (size_t)S * kStage + ExpLoads<4>::kBytes;
};

template <int B, int F>
__device__ __attribute__((always_inline)) inline void read_and_load_exact(const lds_char* __restrict__ rd,
                                                                          lds_char* __restrict__ wr, int kt, int ablk, int bblk,
                                                                          int wave, const Operand<1, false, B, B / 64>& oa,
                                                                          const Operand<1, false, B, B / 64>& ob,
                                                                          const Reader<1, false, B>& rr, u32x4_t (&af)[F],
                                                                          u32x4_t (&bf)[F]) {
    read_stage<B>(rd, ablk, bblk, rr, rr, af, bf);
    __builtin_amdgcn_sched_barrier(0);
    oa.load(wr, wave * (B / 64), kt);
    ob.load(wr + B * 64, wave * (B / 64), kt);
}

template <int B, int S>
__global__ __launch_bounds__(256, 2) void k_mm_fp8_exact(Fp8Args a) {
#ifdef __HIP_DEVICE_COMPILE__          // the host pass needs the signature only
    using L = Exact8<B, S>;
    constexpr int F = L::F;
    extern __shared__ uint4 smem[];
    __shared__ Groups groups;
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), wm = wave >> 1, wn = wave & 1;

    const int w = item_of_block(blockIdx.x, gridDim.x);
    if (w >= count_items<O, B, B, float>(a.m, groups)) return;
    Tile2 t;
    tile_of_item<O, B, B>(a.m, groups, w, t);
    auto oa = operand_a<O, B, L::NL>(a.m, t);
    auto ob = operand_b<O, B, L::NL>(a.m, t);
    oa.plan(wave * L::NL, lane, t.ni);
    ob.plan(wave * L::NL, lane, t.nj);
    const Reader<1, false, B> rr(lane);

    // rows split evenly over the two wavefront rows, in 16-row blocks
    const int half = min(B / 2, (t.ni + 31) / 32 * 16), row0 = uni(wm * half);
    const int nblk = uni(max(0, min(half, t.ni - row0) + 15) / 16);
    f32x4_t acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    const int KT = (t.C + 63) / 64;
    ExpLoads<4> el;
    lds_char* slots = lds + S * L::kStage;
    el.plan(a, t, wave, lane);
    el.load(slots, wave, 0);
#pragma unroll
    for (int q = 0; q < (S - 1) * 2; ++q) {
        oa.load(lds + q * L::kSub, wave * L::NL, q);
        ob.load(lds + q * L::kSub + B * 64, wave * L::NL, q);
    }
    uint32_t ex[F] = {}, ew = 0;
    for (int kt = 0; kt < KT;) {
#pragma unroll
        for (int st = 0; st < S; ++st) {
            if (kt >= KT) break;
            wait_vmcnt<(S - 2) * 2 * 2 * L::NL>();
            lds_barrier();
            if ((kt & 7) == 4) el.load(slots, wave, kt + 4);
            u32x4_t af[2][F], bf[2][F];
            const int nx = (st + S - 1) % S;
#pragma unroll
            for (int u = 0; u < 2; ++u)
                read_and_load_exact<B>(lds + st * L::kStage + u * L::kSub, lds + nx * L::kStage + u * L::kSub,
                                       kt + (S - 1) * 2 + u, row0 / 16, wn * F, wave, oa, ob, rr, af[u], bf[u]);
            if ((kt & 7) == 0) {
                typedef const __attribute__((address_space(3))) uint32_t lds_cu1;
                lds_cu1* s = (lds_cu1*)(slots + ((kt >> 3) & 1) * ExpLoads<4>::kSlot);
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    const int r = min(row0 + 16 * i, B - 16);
                    ex[i] = s[r / 32 * 64 + r % 32 + (lane & 15)];
                }
                ew = s[32];
            }
            wait_lds();
            const int shift = (kt & 6) * 4;
            uint32_t sx[F];
#pragma unroll
            for (int i = 0; i < F; ++i) sx[i] = ex[i] >> shift & 255;
            block_f32(af, bf, sx, ew >> shift & 255, F > 2 ? nblk : F, acc);
            kt += 2;
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");          // no load is left on its way to LDS
#pragma unroll
    for (int i = 0; i < F; ++i) {
        if (i >= nblk) break;
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const int r = row0 + 16 * i + (lane & 15), col = wn * (B / 2) + 16 * j + 4 * (lane >> 4);
            if (r < t.ni && col < t.nj) *reinterpret_cast<f32x4_t*>((float*)a.m.c + (t.crow + r) * a.m.N + t.j0 + col) = acc[i][j];
        }
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

hipError_t launch_fp8_exact(int tile, const Fp8Args& a, hipStream_t st) {
    return tile == 64 ? go<k_mm_fp8_exact<64, 3>, 64>(a, 256, Exact8<64, 3>::kLds, st)
                      : go<k_mm_fp8_exact<128, 2>, 128>(a, 256, Exact8<128, 2>::kLds, st);
}

}  // namespace moe
