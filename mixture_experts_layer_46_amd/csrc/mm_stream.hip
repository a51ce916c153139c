// Weight gradients of groups of middling size in large tiles (kind 2 of mm_tile.h, bf16):
// 256 x 256 on the matrix cores.
//
// The contractions, a group's rows, are short, so that what stands between two tiles counts.
// The grid is persistent and the steps of a workgroup's tiles form one stream: the last four
// steps of a tile load the first four stages of the next, and between two tiles stand the
// output and one table look-up.  Within a step a wavefront multiplies the operands it holds in
// registers, reads the next step's from LDS and starts the loads of the fourth step after,
// spread between the matrix instructions; one barrier a step.  (mm.hip's two groups half a
// step apart are faster step by step, but its tiles share no loads.)
#include "mm_large.h"

namespace moe {

namespace {

using namespace large;
using O = Op<2, Elem::bf16>;

constexpr int kCS = kT + 8;                   // bf16 per row of the output piece
constexpr size_t kLds = (size_t)kStages * kStage + 32 * kCS * 2;      // stages; 32 rows on their way out

// One step: the products of the operands in registers, with the next step's operands read
// from stage `rd` and a later step's loads started into stage `wr` in between (two reads
// after each of six row blocks, the loads after the third and the fifth: measured against
// denser and later placements, 1-4% on the large shapes).  The matrix instruction takes the
// B operand first, so that a lane's four sums are four columns of one row.
// The stages are separate __restrict__ arguments: otherwise the compiler takes the
// transposing reads to touch what is in flight, and waits for every load before them.
__device__ __attribute__((always_inline)) inline void step(const lds_char* __restrict__ rd, lds_char* __restrict__ wr,
                                                           int kload, int nblk, int wm, int wn, int wave,
                                                           const OpA<O>& oa, const OpB<O>& ob,
                                                           const Reader<O::ES, O::kACols, kT>& ra,
                                                           const Reader<O::ES, O::kBCols, kT>& rb,
                                                           const u32x4_t (&af)[8], const u32x4_t (&bf)[4],
                                                           u32x4_t (&an)[8], u32x4_t (&bn)[4],
                                                           O::Acc (&acc)[8][4]) {
    asm volatile("" : "+s"(nblk));    // compared anew at each row block (a scalar compare; kept masks cost vector ones)
    wait_lds();                       // this step's operands are in registers: their stage is free
    wait_vmcnt<kVmcnt>();             // this wavefront's loads of the next step have landed
    lds_barrier();                    // everyone's
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (__builtin_expect(i < nblk, 1)) {                  // a full tile falls through
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = mma<O::ELEM>(bf[j], af[i], acc[i][j]);
        }
#pragma unroll
        for (int q = 2 * i; q < 2 * i + 2; ++q) {
            if (q < 4) bn[q] = rb(rd + kT * 64, wn * 4 + q);
            else if (q < 12) an[q - 4] = ra(rd, wm * 8 + q - 4);
        }
        if (i == 2) oa.load(wr, wave * kLoads, kload);
        if (i == 4) ob.load(wr + kT * 64, wave * kLoads, kload);
    }
    // the sums live in accumulator registers, next to the two sets of operands
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[i][j]));
}

// A finished tile, one rounding.  Lane l holds row l & 15 and columns 4 (l >> 4) .. + 3 of each
// 16 x 16 block.  bf16 goes out in whole rows of 512 bytes: 16 rows of the upper and 16 of the
// lower wavefronts at a time, through a piece of LDS beside the stages, which the next tile's
// loads are filling.  (Stores straight from registers, 64 bytes of a row at a time, took 8 us
// more for the 32 MB that the tiles of 4096 x 4096 write at once.  Letting the next tile's
// first steps not wait for the stores, which the counter of the loads also counts, cost the
// steps more than it saved: 151 -> 156 us at 256 rows a group.)
template <typename OUT>
__device__ __forceinline__ void store_tile(const MmArgs& a, const Tile2& t, lds_char* piece, int nblk, int wm, int wn,
                                           const O::Acc (&acc)[8][4]) {
    const int rounds = uni((min(t.ni, 128) + 15) / 16);
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));             // what follows is computed here, not kept through the steps
    const int l16 = tid & 15, lq = (tid & 63) >> 4;
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(3))) u32x2_t lds_u2;
    typedef __attribute__((address_space(3))) u32x4_t lds_u4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= rounds) break;               // the same for every wavefront: the barriers match
        if constexpr (sizeof(OUT) == 2) {
            wait_lds();
            lds_barrier();                    // the round before has been read
            if (i < nblk) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *(lds_u2*)(piece + ((wm * 16 + l16) * kCS + wn * 64 + 16 * j + 4 * lq) * 2) =
                        u32x2_t{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
            }
            wait_lds();
            lds_barrier();
#pragma unroll
            for (int q = 0; q < 2; ++q) {     // half q: 16 rows of the wavefronts wm = q, 32 threads a row
                const int rr = (tid >> 5) & 15, c = (tid & 31) * 8, r = q * 128 + 16 * i + rr;
                if (r < t.ni && c < t.nj)
                    __builtin_nontemporal_store(*(const lds_u4*)(piece + ((q * 16 + rr) * kCS + c) * 2),
                                                reinterpret_cast<u32x4_t*>((bf16_t*)a.c + (t.crow + r) * a.N + t.j0 + c));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = wm * 128 + 16 * i + l16, c = wn * 64 + 16 * j + 4 * lq;
                if (r < t.ni && c < t.nj) *reinterpret_cast<f32x4_t*>((float*)a.c + (t.crow + r) * a.N + t.j0 + c) = acc[i][j];
            }
        }
    }
}

template <typename OUT>
__global__ __launch_bounds__(512, 1) void k_mm_stream(MmArgs a) {
#ifdef __HIP_DEVICE_COMPILE__          // the host pass needs the signature only
    extern __shared__ uint4 smem[];
    __shared__ Groups groups;
    lds_char* lds = (lds_char*)smem;
    const int lane = threadIdx.x & 63, wave = uni((int)threadIdx.x >> 6), wm = wave >> 2, wn = wave & 3;
    const Reader<O::ES, O::kACols, kT> ra(lane);
    const Reader<O::ES, O::kBCols, kT> rb(lane);

    // this workgroup's item in round r; the last, partial round is dealt block by block
    const int total = count_items<O, kT, kT, OUT>(a, groups), G = gridDim.x;
    auto item = [&](int r) {
        const int left = total - r * G;
        const int i = left >= G ? item_of_block(blockIdx.x, G) : (int)blockIdx.x;
        return i < left ? r * G + i : -1;
    };
    // A tile takes an even number of steps (two are unrolled), at least four, so that its last
    // four always load the next tile's first; steps past the contraction multiply the zeros
    // that their loads read.
    auto steps_of = [](const Tile2& t) { return max(4, ((t.C + O::kStep - 1) / O::kStep + 1) & ~1); };
    OpA<O> oa;
    OpB<O> ob;
    auto load_from = [&](const Tile2& t) {
        oa = operand_a<O, kT, kLoads>(a, t);
        ob = operand_b<O, kT, kLoads>(a, t);
        int l = lane;
        asm volatile("" : "+v"(l));           // the offsets are computed here, not their parts kept
        oa.plan(wave * kLoads, l, t.ni);
        ob.plan(wave * kLoads, l, t.nj);
    };

    int round = 0;
    if (item(0) < 0) return;
    Tile2 cur, nxt;
    tile_of_item<O, kT, kT>(a, groups, item(0), cur);
    load_from(cur);
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
        oa.load(lds + s * kStage, wave * kLoads, s);
        ob.load(lds + s * kStage + kT * 64, wave * kLoads, s);
    }
    wait_vmcnt<3 * 2 * kLoads>();             // the first step's stage; from here on each step waits for the next one's
    lds_barrier();
    int g = 0;                                // steps so far: step g reads stage g mod 4
    for (;;) {
        O::Acc acc[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = O::Acc{0, 0, 0, 0};
        u32x4_t a0[8], b0[4], a1[8], b1[4];
        read_stage<kT>(lds + (g & 3) * kStage, wm * 8, wn * 4, ra, rb, a0, b0);
        const int KT = steps_of(cur), nblk = uni(max(0, min(128, cur.ni - wm * 128) + 15) / 16);
        int next = -1;
        for (int kt = 0, kload = 4; kt < KT; kt += 2, kload += 2, g += 2) {
            if (kload == KT) {                // the loads pass on to the next tile
                next = item(++round);
                if (next >= 0) {
                    tile_of_item<O, kT, kT>(a, groups, next, nxt);
                    load_from(nxt);
                    kload = 0;
                }
            }
            lds_char *s0 = lds + (g & 3) * kStage, *s1 = lds + ((g + 1) & 3) * kStage, *s2 = lds + ((g + 2) & 3) * kStage;
            step(s1, s0, kload, nblk, wm, wn, wave, oa, ob, ra, rb, a0, b0, a1, b1, acc);
            step(s2, s1, kload + 1, nblk, wm, wn, wave, oa, ob, ra, rb, a1, b1, a0, b0, acc);
        }
        store_tile<OUT>(a, cur, lds + kStages * kStage, nblk, wm, wn, acc);
        if (next < 0) break;
        cur = nxt;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");          // no load is left on its way to LDS
#endif
}

template <typename OUT>
hipError_t go(const MmArgs& a, hipStream_t st) {
    const hipError_t e = allow_lds<k_mm_stream<OUT>>(kLds);
    if (e != hipSuccess) return e;
    const long long items = mm_blocks(a, O::KIND, kT, kT), cus = device_cu_count();
    hipLaunchKernelGGL((k_mm_stream<OUT>), dim3((unsigned)(items < cus ? items : cus)), dim3(512), kLds, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mm_stream(int out_dtype, const MmArgs& a, hipStream_t st) {
    return out_dtype == MOE_F32 ? go<float>(a, st) : go<bf16_t>(a, st);
}

}  // namespace moe
