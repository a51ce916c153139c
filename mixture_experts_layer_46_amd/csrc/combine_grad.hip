// Gradient of the gate-weighted combine out[t] = sum_j w[t, j] y_perm[row(t, j)]:
//   dy_perm[row(t, j)] = w[t, j] dout[t]          dw[t, j] = <dout[t], y_perm[row(t, j)]>
// A dropped pair (row -1) has no grouped row and dw = 0.  One workgroup per token: its
// output gradient is read once for all k rows, each grouped row is read and written once.
// The dot products are summed in fp32 in a fixed order (per lane, then across the lanes of
// a wavefront, then the wavefronts), so results do not depend on scheduling.
// Rows are written with the non-temporal hint, and read with it where y_perm exceeds the
// 256 MB that the memory-side cache holds (8192 tokens of 8 experts, 7168 wide: 407 -> 382 us,
// 5.2 TB/s; 8192 of 2, 4096 wide: 67 -> 50.5 us, with the hint on the reads too 57).
#include "common.h"
#include "launch.h"
#include "mm_launch.h"

namespace moe {

namespace {

template <bool BF16>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (BF16) f[2 * q] = bf16lo_to_f32(d[q]), f[2 * q + 1] = bf16hi_to_f32(d[q]);
        else f[q] = __uint_as_float(d[q]);
    }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    if constexpr (BF16)
        return uint4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
    else
        return uint4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
}

// P threads per token: a workgroup, or for short rows one wavefront (4 tokens a workgroup).
template <bool BF16, int P, bool NT>
__global__ __launch_bounds__(256) void k_combine_grad(const uint4* __restrict__ dout, const uint4* __restrict__ y,
                                                      const int32_t* __restrict__ row_of_pair,
                                                      const float* __restrict__ w, uint4* __restrict__ dy,
                                                      float* __restrict__ dw, long long T, int k, int chunks, int rows) {
    constexpr int NV = BF16 ? 8 : 4;
    __shared__ float part[4][8];
    const long long t = (long long)blockIdx.x * (256 / P) + threadIdx.x / P;
    if (P == 64 && t >= T) return;                     // a whole wavefront
    int row[8];
    float g[8], dot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        row[j] = j < k ? row_of_pair[t * k + j] : -1;
        if (row[j] >= rows) row[j] = -1;
        g[j] = j < k ? w[t * k + j] : 0.f;
        dot[j] = 0.f;
    }
    for (int c = threadIdx.x % P; c < chunks; c += P) {
        float d[8];
        unpack<BF16>(dout[t * chunks + c], d);
        uint4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (row[j] >= 0) {
                const u32x4_t* p = reinterpret_cast<const u32x4_t*>(y + (long long)row[j] * chunks + c);
                v[j] = __builtin_bit_cast(uint4, NT ? __builtin_nontemporal_load(p) : *p);
            }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (row[j] < 0) continue;
            float f[8], o[8];
            unpack<BF16>(v[j], f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                dot[j] = fmaf(d[i], f[i], dot[j]);
                o[i] = g[j] * d[i];
            }
            __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, pack<BF16>(o)),
                                        reinterpret_cast<u32x4_t*>(dy + (long long)row[j] * chunks + c));
        }
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j >= k) break;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) dot[j] += __shfl_xor(dot[j], off);
        if constexpr (P > 64) {
            if (lane == 0) part[wave][j] = dot[j];
        } else {
            if (lane == j) dw[t * k + j] = dot[j];
        }
    }
    if constexpr (P > 64) {
        __syncthreads();
        if ((int)threadIdx.x < k) {
            const int j = threadIdx.x;
            dw[t * k + j] = ((part[0][j] + part[1][j]) + part[2][j]) + part[3][j];
        }
    }
}

template <bool BF16>
void go(const void* dout, const void* y_perm, const int32_t* row_of_pair, const float* w, void* dy_perm, float* dw,
        long long T, int k, int chunks, long long rows, hipStream_t st) {
    auto run = [&](auto kern, int p) {
        hipLaunchKernelGGL(kern, dim3((unsigned)((T * p + 255) / 256)), dim3(256), 0, st, (const uint4*)dout,
                           (const uint4*)y_perm, row_of_pair, w, (uint4*)dy_perm, dw, T, k, chunks, (int)rows);
    };
    const bool nt = rows * chunks * 16 > (256ll << 20);
    if (chunks <= 128) nt ? run(k_combine_grad<BF16, 64, true>, 64) : run(k_combine_grad<BF16, 64, false>, 64);
    else nt ? run(k_combine_grad<BF16, 256, true>, 256) : run(k_combine_grad<BF16, 256, false>, 256);
}

}  // namespace

hipError_t launch_combine_grad(const void* dout, const void* y_perm, const int32_t* row_of_pair, const float* w,
                               void* dy_perm, float* dw, long long T, int k, int H, int dtype, long long rows,
                               hipStream_t st) {
    if (dtype == MOE_BF16) go<true>(dout, y_perm, row_of_pair, w, dy_perm, dw, T, k, H / 8, rows, st);
    else go<false>(dout, y_perm, row_of_pair, w, dy_perm, dw, T, k, H / 4, rows, st);
    return hipGetLastError();
}

}  // namespace moe
