// What the two kernels of the large tiles share (mm.hip, mm_stream.hip): 256 x 256 tiles by
// eight wavefronts, 2 x 4 over the tile: 128 x 64 wavefront tiles of 128 accumulator
// registers, two wavefronts per SIMD; operands in four LDS stages of 32 KB.
#pragma once

#include "mm_tile.h"

namespace moe {
namespace large {

constexpr int kT = 256;                       // tile rows and columns
constexpr int kStage = 2 * kT * 64;           // bytes of a step: the A operand, then the B operand
constexpr int kStages = 4;
constexpr int kLoads = 2;                     // loads of one operand per wavefront and step
constexpr int kVmcnt = 4 * kLoads;            // loads of the two steps after the awaited one


template <typename O>
using OpA = Operand<O::ES, O::kACols, kT, kLoads>;
template <typename O>
using OpB = Operand<O::ES, O::kBCols, kT, kLoads>;

// One step: the products of the operands in registers, with the next step's operands read
// from stage `rd` and a later step's loads started into stage `wr` in between (two reads
// after each of six row blocks, the loads after the third and the fifth: measured against
// denser and later placements, 1-4% on the large shapes).  The matrix instruction takes the
// B operand first, so that a lane's four sums are four columns of one row.
// The stages are separate __restrict__ arguments: otherwise the compiler takes the
// transposing reads to touch what is in flight, and waits for every load before them.
template <typename O>
__device__ __attribute__((always_inline)) inline void step(const lds_char* __restrict__ rd, lds_char* __restrict__ wr,
                                                           int kload, int nblk, int wm, int wn, int wave,
                                                           const OpA<O>& oa, const OpB<O>& ob,
                                                           const Reader<O::ES, O::kACols, kT>& ra,
                                                           const Reader<O::ES, O::kBCols, kT>& rb,
                                                           const u32x4_t (&af)[8], const u32x4_t (&bf)[4],
                                                           u32x4_t (&an)[8], u32x4_t (&bn)[4],
                                                           typename O::Acc (&acc)[8][4]) {
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

}  // namespace large
}  // namespace moe
