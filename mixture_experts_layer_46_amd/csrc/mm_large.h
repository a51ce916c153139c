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
using OpA = OperandA<O, kT, kLoads>;
template <typename O>
using OpB = OperandB<O, kT, kLoads>;

}  // namespace large
}  // namespace moe
