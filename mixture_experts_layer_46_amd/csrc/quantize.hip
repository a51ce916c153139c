// Quantisation to 8-bit integers: rows (a scale per token) and expert weights (a scale per
// expert and output channel).
//
//   scale = amax / 127 (fp32, one rounding),  q = x / scale to the nearest integer, ties to
//   even, of the exact ratio: the fp32 quotient decides, and where it lies on the border
//   between two integers the exact remainder x - q scale (one fma) corrects it.
// A row or channel of zeros has scale 0 and q 0.  One that holds an infinity or a NaN has
// scale NaN and q 0, so that what is computed from it is NaN, not a wrong number.
#include "common.h"
#include "launch.h"
#include "mm_launch.h"

namespace moe {

namespace {

__device__ __forceinline__ int quant1(float x, float s) {
    float q = rintf(x / s);
    const float r = fmaf(-q, s, x);                    // exact: |r| <= s (1/2 + 2^-17)
    if (2.f * fabsf(r) > s) q += r > 0.f ? 1.f : -1.f;
    return (int)fminf(fmaxf(q, -127.f), 127.f);        // a subnormal scale may round the ratio past 127
}
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
    const float s = __uint_as_float(amax_bits) / 127.f;
    return amax_bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : s;
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// 8 consecutive elements as fp32
__device__ __forceinline__ void get8(const bf16_t* p, float (&v)[8]) {
    const uint4 d = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) v[2 * q] = bf16lo_to_f32(w[q]), v[2 * q + 1] = bf16hi_to_f32(w[q]);
}
__device__ __forceinline__ void get8(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// One workgroup per row: the row's largest magnitude, then its integers (the second read
// comes from the caches).
template <typename T>
__global__ __launch_bounds__(256) void k_quantize_rows(const T* __restrict__ x, int K, int8_t* __restrict__ q,
                                                       float* __restrict__ scale) {
    __shared__ uint32_t part[4];
    const long long r = blockIdx.x;
    const T* xr = x + r * K;
    uint32_t m = 0;
    for (int c = threadIdx.x * 8; c < K; c += 2048) {
        float v[8];
        get8(xr + c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    const float s = scale_of(max(max(part[0], part[1]), max(part[2], part[3])));
    if (threadIdx.x == 0) scale[r] = s;
    for (int c = threadIdx.x * 8; c < K; c += 2048) {
        float v[8];
        get8(xr + c, v);
        uint32_t w[2] = {0u, 0u};
        if (s > 0.f)
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j >> 2] |= (uint32_t)(quant1(v[j], s) & 0xff) << (8 * (j & 3));
        *reinterpret_cast<uint2*>(q + r * K + c) = uint2{w[0], w[1]};
    }
}

// Expert weights [E, K, N] -> q [E, N, K], scale [E, N].  One workgroup per expert and 64
// output channels: the channels' largest magnitudes over K, then 64 x 64 blocks through
// LDS, so that both the reads (along N) and the writes (along K) are contiguous.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize_experts(const T* __restrict__ w, int K, int N,
                                                          int8_t* __restrict__ q, float* __restrict__ scale) {
    __shared__ uint32_t mx[64];
    __shared__ float sc[64];
    __shared__ int8_t tile[64][80];                    // [channel][k], rows of 80 bytes
    const int e = blockIdx.y, n0 = blockIdx.x * 64, tid = threadIdx.x;
    const T* we = w + (long long)e * K * N;
    const int c8 = (tid & 7) * 8, kr = tid >> 3;       // 8 channels of one of 32 rows
    if (tid < 64) mx[tid] = 0;
    __syncthreads();
    uint32_t m[8] = {};
    if (n0 + c8 < N)
        for (int k = kr; k < K; k += 32) {
            float v[8];
            get8(we + (long long)k * N + n0 + c8, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = max(m[j], abs_bits(v[j]));
        }
#pragma unroll
    for (int j = 0; j < 8; ++j) atomicMax(&mx[c8 + j], m[j]);
    __syncthreads();
    if (tid < 64) {
        sc[tid] = scale_of(mx[tid]);
        if (n0 + tid < N) scale[(long long)e * N + n0 + tid] = sc[tid];
    }
    __syncthreads();
    for (int k0 = 0; k0 < K; k0 += 64) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = k0 + kr + 32 * h;
            float v[8] = {};
            if (n0 + c8 < N && k < K) get8(we + (long long)k * N + n0 + c8, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float s = sc[c8 + j];
                tile[c8 + j][kr + 32 * h] = s > 0.f ? (int8_t)quant1(v[j], s) : (int8_t)0;
            }
        }
        __syncthreads();
        const int n = tid >> 2, kc = (tid & 3) * 16;   // K is a multiple of 16
        if (n0 + n < N && k0 + kc < K)
            *reinterpret_cast<uint4*>(q + ((long long)e * N + n0 + n) * K + k0 + kc) =
                *reinterpret_cast<const uint4*>(&tile[n][kc]);
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_quantize_rows(const void* x, int dtype, long long rows, int K, int8_t* q, float* scale,
                                hipStream_t st) {
    const dim3 g((unsigned)rows), t(256);
    if (dtype == MOE_BF16) hipLaunchKernelGGL(k_quantize_rows<bf16_t>, g, t, 0, st, (const bf16_t*)x, K, q, scale);
    else hipLaunchKernelGGL(k_quantize_rows<float>, g, t, 0, st, (const float*)x, K, q, scale);
    return hipGetLastError();
}

hipError_t launch_quantize_experts(const void* w, int dtype, int E, int K, int N, int8_t* q, float* scale,
                                   hipStream_t st) {
    const dim3 g((N + 63) / 64, E), t(256);
    if (dtype == MOE_BF16) hipLaunchKernelGGL(k_quantize_experts<bf16_t>, g, t, 0, st, (const bf16_t*)w, K, N, q, scale);
    else hipLaunchKernelGGL(k_quantize_experts<float>, g, t, 0, st, (const float*)w, K, N, q, scale);
    return hipGetLastError();
}

}  // namespace moe
