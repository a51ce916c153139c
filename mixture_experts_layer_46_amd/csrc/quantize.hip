// Quantisation to 8-bit integers: rows (a scale per token) and expert weights (a scale per
// expert and output channel).
//
//   scale = amax / 127 (fp32, one rounding),  q = x / scale to the nearest integer, ties to
//   even, of the exact ratio.  x times the scale's reciprocal is within 2^-16 of the ratio and
//   rounds to q except next to a border between two integers; the remainder x - q scale, which
//   one fma gives exactly, shows those cases (at least half a scale), and they take the
//   quotient instead.  The kernel then keeps up with memory: 8192 x 4096 bf16 26 us with a
//   division for every element.
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

// Eight integers of v, packed.  Adding 1.5 2^23 rounds to an integer (ties to even) and
// leaves it in the low bits.
__device__ __forceinline__ uint2 quant8(const float (&v)[8], float s, float inv) {
    constexpr float kMagic = 12582912.f;
    uint32_t b[8];
    bool border = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = fmaf(v[j], inv, kMagic), q = t - kMagic;
        border |= !(fabsf(fmaf(-q, s, v[j])) * 2.f < s);
        b[j] = __float_as_uint(t);
    }
    if (__builtin_expect(border, 0))
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = (uint32_t)quant1(v[j], s);
    auto pack4 = [](const uint32_t* p) {
        const uint32_t lo = __builtin_amdgcn_perm(p[1], p[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(p[3], p[2], 0x0c0c0400u);
        return lo | hi << 16;
    };
    return uint2{pack4(b), pack4(b + 4)};
}

// P threads per row (16, a wavefront, or a workgroup for long rows); the row's first P * C
// chunks of 8 elements stay in registers between the largest magnitude and the integers, so
// rows up to that length are read once.
template <typename T, int P, int C>
__global__ __launch_bounds__(256) void k_quantize_rows(const T* __restrict__ x, long long rows, int K,
                                                       int8_t* __restrict__ q, float* __restrict__ scale) {
    __shared__ uint32_t part[4];
    const long long r = (long long)blockIdx.x * (256 / P) + threadIdx.x / P;
    const bool live = r < rows;                        // P < 64: the last wavefront's rows may end inside it
    const int t = threadIdx.x % P;
    const T* xr = x + r * K;
    int8_t* qr = q + r * K;
    float v[C][8];
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = (c * P + t) * 8;
        if (live && k < K) {
            get8(xr + k, v[c]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[c][j] = 0.f;
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[c][j]));
    for (int k = (C * P + t) * 8; live && k < K; k += P * 8) {
        float u[8];
        get8(xr + k, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(u[j]));
    }
#pragma unroll
    for (int off = (P < 64 ? P : 64) / 2; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off));
    if constexpr (P > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
        __syncthreads();
        m = max(max(part[0], part[1]), max(part[2], part[3]));
    }
    if (!live) return;
    const float s = scale_of(m);
    if (t == 0) scale[r] = s;
    // a scale whose reciprocal could overflow (subnormal rows): quotients throughout
    const bool plain = s >= 0x1p-120f;
    const float inv = 1.f / s;
    auto put = [&](int k, const float (&u)[8]) {
        uint2 w{0u, 0u};
        if (plain) {
            w = quant8(u, s, inv);
        } else if (s > 0.f) {
            uint32_t b[2] = {0u, 0u};
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j >> 2] |= (uint32_t)(quant1(u[j], s) & 0xff) << (8 * (j & 3));
            w = uint2{b[0], b[1]};
        }
        *reinterpret_cast<uint2*>(qr + k) = w;
    };
#pragma unroll
    for (int c = 0; c < C; ++c)
        if ((c * P + t) * 8 < K) put((c * P + t) * 8, v[c]);
    for (int k = (C * P + t) * 8; k < K; k += P * 8) {
        float u[8];
        get8(xr + k, u);
        put(k, u);
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
    __shared__ alignas(16) int8_t tile[64][80];        // [channel][k], rows of 80 bytes
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

namespace {

template <typename T>
void rows_of(const void* x, long long rows, int K, int8_t* q, float* scale, hipStream_t st) {
    auto run = [&](auto kern, int p) {
        hipLaunchKernelGGL(kern, dim3((unsigned)((rows * p + 255) / 256)), dim3(256), 0, st, (const T*)x, rows, K, q, scale);
    };
    // the fewest threads that hold the row in 4 (at last 8) chunks each
    if (K <= 512) run(k_quantize_rows<T, 16, 4>, 16);
    else if (K <= 2048) run(k_quantize_rows<T, 64, 4>, 64);
    else if (K <= 8192) run(k_quantize_rows<T, 256, 4>, 256);
    else run(k_quantize_rows<T, 256, 8>, 256);
}

}  // namespace

hipError_t launch_quantize_rows(const void* x, int dtype, long long rows, int K, int8_t* q, float* scale,
                                hipStream_t st) {
    if (dtype == MOE_BF16) rows_of<bf16_t>(x, rows, K, q, scale, st);
    else rows_of<float>(x, rows, K, q, scale, st);
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
