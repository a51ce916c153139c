// The sigmoid of the experts' activation (dropout.hip, mm_tile.h).
#pragma once

#include "common.h"

namespace moe {

// exp(x) for x <= 0 by the hardware's base-2 exponential, which flushes subnormal results:
// below 2^-126 it is taken 2^64 higher and scaled back.
__device__ __forceinline__ float fast_exp(float x) {
    const float y = x * 1.44269504f;
    const bool tiny = y < -126.f;
    const float r = __builtin_amdgcn_exp2f(tiny ? y + 64.f : y);
    return tiny ? r * 0x1p-64f : r;
}

// s = 1 / (1 + exp(-a)) and 1 - s, both without cancellation or overflow.  bf16 results
// take the hardware's exponential and reciprocal.  The fp32 product a log2(e) puts up to
// 1.25 |a| 2^-24 on the exponential's relative error (2^-17 where it reaches the least normal
// value), beside a few 2^-23 of the two instructions: far below the results' own 2^-9.
template <bool FAST>
__device__ __forceinline__ void sigmoid(float a, float& s, float& ns) {
    const float t = FAST ? fast_exp(-fabsf(a)) : expf(-fabsf(a));
    const float big = FAST ? __builtin_amdgcn_rcpf(1.f + t) : 1.f / (1.f + t), small = t * big;
    s = a >= 0.f ? big : small;
    ns = a >= 0.f ? small : big;
}

}  // namespace moe
