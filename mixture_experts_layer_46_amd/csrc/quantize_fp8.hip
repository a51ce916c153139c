// Quantisation to 8-bit floating point (e4m3) with a power-of-two scale for each block: 128
// consecutive elements of a row, or 128 x 128 of an expert matrix.
//
//   scale = 2^e, the least e >= -127 for which the block's largest magnitude is at most 448 2^e;
//   q = x 2^-e to the nearest e4m3 number, ties to even.
//
// With amax = m 2^k, 1 <= m < 2, that is e = k - 8, or k - 7 where m > 1.75 (448 = 1.75 2^8): the
// biased exponent and one compare of the mantissa.  x 2^-e is exact but for numbers far below
// e4m3's smallest, so that q is rounded once.  The scale is held as e + 127 in a byte.  A block
// with an infinity or a NaN gets the byte 255, which the product's instruction takes for NaN,
// and q 0.  A row of scales is padded to a multiple of 4 bytes (so that a product reads four at
// once); padding is 127 (a scale of 1).
//
// Memory bounds both kernels.  Rows: 65536 x 7168 bf16 248 us (5.7 TB/s), 8192 x 4096 bf16 20 us
// (5.0).  Experts, which the weights' layout asks to be transposed: 64 of 4096 x 1408 210 us (5.3).
#include "common.h"
#include "launch.h"
#include "mm_fp8.h"
#include "mm_launch.h"

namespace moe {

namespace {

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t exponent_of(uint32_t amax) {
    const int e = (int)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return amax >= 0x7f800000u ? 255u : (uint32_t)max(e, 0);
}
// 2^(127 - byte), which brings the block into e4m3's range; 0 for a block that is not finite
__device__ __forceinline__ float factor_of(uint32_t byte) { return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23); }

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
__device__ __forceinline__ uint32_t max8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
    return m;
}
// Eight numbers times f (a power of two, or 0: then zeros, whatever v holds).
__device__ __forceinline__ uint2 pack8(const float (&v)[8], float f) {
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = f == 0.f ? 0.f : v[j] * f;
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false), hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[4], s[5], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[6], s[7], hi, true);
    return uint2{(uint32_t)lo, (uint32_t)hi};
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t max16(uint32_t x) {        // over each 16 lanes, in all of them
    x = dpp_max<0xB1>(x);
    x = dpp_max<0x4E>(x);
    x = dpp_max<0x141>(x);
    return dpp_max<0x140>(x);
}

// A wavefront takes 512 elements of a row at a time: four blocks of 16 lanes x 8, and their four
// bytes.  W wavefronts share a row; a wavefront has C loads in flight.  Memory bounds it.
template <typename T, int W, int C>
__global__ __launch_bounds__(256) void k_quantize_rows_fp8(const T* __restrict__ x, long long rows, int K,
                                                           uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, chunks = (K + 511) / 512;
    const long long r = (long long)blockIdx.x * (4 / W) + wave / W;
    if (r >= rows) return;
    for (int c0 = wave % W; c0 < chunks; c0 += W * C) {
        float v[C][8];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int k = (c0 + i * W) * 512 + lane * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
            if (k < K) get8(x + r * K + k, v[i]);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = c0 + i * W, k = c * 512 + lane * 8;
            if (c >= chunks) break;
            uint32_t b = exponent_of(max16(max8(v[i])));
            if (k < K) *reinterpret_cast<uint2*>(q + r * K + k) = pack8(v[i], factor_of(b));
            if ((k & ~127) >= K) b = 127u;                      // padding
            const uint32_t b0 = __builtin_amdgcn_readlane(b, 0), b1 = __builtin_amdgcn_readlane(b, 16),
                           b2 = __builtin_amdgcn_readlane(b, 32), b3 = __builtin_amdgcn_readlane(b, 48);
            if (lane == 0)
                *reinterpret_cast<uint32_t*>(scale + r * (4ll * chunks) + 4 * c) = b0 | b1 << 8 | b2 << 16 | b3 << 24;
        }
    }
}

// Rows of at most B = 1 or 2 blocks: 4 / B of them to a wavefront, which has two such sets in flight.
// 100000 x 256 bf16 15 us (5.2 TB/s; a row to a wavefront 22), 60000 x 128 bf16 8 us, the host's call.
template <typename T, int B>
__global__ __launch_bounds__(256) void k_quantize_short_rows_fp8(const T* __restrict__ x, long long rows, int K,
                                                                 uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
    constexpr int C = 2, RW = 4 / B;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, blk = lane >> 4, k = blk % B * 128 + (lane & 15) * 8;
    const long long r0 = ((long long)blockIdx.x * 4 + wave) * (C * RW) + blk / B;
    float v[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        if (r0 + i * RW < rows && k < K) get8(x + (r0 + i * RW) * K + k, v[i]);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const long long r = r0 + i * RW;
        const uint32_t b = exponent_of(max16(max8(v[i])));
        const bool live = r < rows;
        if (live && k < K) *reinterpret_cast<uint2*>(q + r * K + k) = pack8(v[i], factor_of(b));
        uint32_t pad = 127u;                                  // the second block's byte
        if constexpr (B == 2) {
            const uint32_t up = lane < 32 ? __builtin_amdgcn_readlane(b, 16) : __builtin_amdgcn_readlane(b, 48);
            if (K > 128) pad = up;
        }
        if (live && lane % (16 * B) == 0) *reinterpret_cast<uint32_t*>(scale + r * 4) = b | pad << 8 | 0x7f7f0000u;
    }
}

// One block of 128 x 128 of w [E, K, N] per workgroup, read once, transposed through LDS into
// q [E, N, K] as whole lines.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize_experts_fp8(const T* __restrict__ w, int K, int N, uint8_t* __restrict__ q,
                                                              uint8_t* __restrict__ scale) {
    constexpr int kRow = 144;                                 // bytes of an LDS row: 128 and padding against bank conflicts
    __shared__ uint4 tile4[128 * kRow / 16];
    __shared__ uint32_t part[4];
    uint8_t* tile = reinterpret_cast<uint8_t*>(tile4);
    const int tid = threadIdx.x, KB = (K + 127) / 128, NB = (N + 127) / 128, sb = fp8_scale_bytes(K);
    const int kb = blockIdx.x % KB, nb = (int)((blockIdx.x / KB) % NB), e = (int)(blockIdx.x / KB / NB);
    const int k0 = kb * 128 + tid / 16 * 8, n0 = nb * 128 + tid % 16 * 8;      // this thread's 8 x 8
    float v[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        if (k0 + i < K && n0 < N) get8(w + ((long long)e * K + k0 + i) * N + n0, v[i]);
        m = max(m, max8(v[i]));
    }
    m = max16(m);
    const uint32_t wm = max(max((uint32_t)__builtin_amdgcn_readlane(m, 0), (uint32_t)__builtin_amdgcn_readlane(m, 16)),
                            max((uint32_t)__builtin_amdgcn_readlane(m, 32), (uint32_t)__builtin_amdgcn_readlane(m, 48)));
    if ((tid & 63) == 0) part[tid >> 6] = wm;
    __syncthreads();
    const uint32_t b = exponent_of(max(max(part[0], part[1]), max(part[2], part[3])));
    const float f = factor_of(b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float col[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) col[i] = v[i][j];
        *reinterpret_cast<uint2*>(tile + (tid % 16 * 8 + j) * kRow + tid / 16 * 8) = pack8(col, f);
    }
    __syncthreads();
    for (int c = tid; c < 128 * 8; c += 256) {
        const int n = c / 8, k = (c % 8) * 16;
        if (nb * 128 + n < N && kb * 128 + k < K)
            *reinterpret_cast<uint4*>(q + ((long long)e * N + nb * 128 + n) * K + kb * 128 + k) =
                *reinterpret_cast<const uint4*>(tile + n * kRow + k);
    }
    uint8_t* s = scale + ((long long)e * NB + nb) * sb;
    if (tid == 0) s[kb] = (uint8_t)b;
    if (kb == KB - 1)
        for (int i = KB + tid; i < sb; i += 256) s[i] = 127;
}

template <typename T>
hipError_t rows(const T* x, long long n, int K, uint8_t* q, uint8_t* scale, hipStream_t st) {
    const int chunks = (K + 511) / 512;
#define GO(W, C) \
    hipLaunchKernelGGL((k_quantize_rows_fp8<T, W, C>), dim3((unsigned)((n + 4 / W - 1) / (4 / W))), dim3(256), 0, st, x, n, K, q, scale)
    if (K <= 256) {
        const dim3 grid((unsigned)(K <= 128 ? (n + 31) / 32 : (n + 15) / 16));
        if (K <= 128) hipLaunchKernelGGL((k_quantize_short_rows_fp8<T, 1>), grid, dim3(256), 0, st, x, n, K, q, scale);
        else hipLaunchKernelGGL((k_quantize_short_rows_fp8<T, 2>), grid, dim3(256), 0, st, x, n, K, q, scale);
    } else if (chunks <= 1) GO(1, 1);
    else if (chunks <= 2) GO(1, 2);
    else if (chunks <= 4) GO(2, 2);
    else GO(4, 2);
#undef GO
    return hipGetLastError();
}

template <typename T>
hipError_t experts(const T* w, int E, int K, int N, uint8_t* q, uint8_t* scale, hipStream_t st) {
    const long long blocks = (long long)E * ((K + 127) / 128) * ((N + 127) / 128);
    hipLaunchKernelGGL(k_quantize_experts_fp8<T>, dim3((unsigned)blocks), dim3(256), 0, st, w, K, N, q, scale);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows_fp8(const void* x, int dtype, long long n, int K, uint8_t* q, uint8_t* scale, hipStream_t st) {
    return dtype == MOE_F32 ? rows((const float*)x, n, K, q, scale, st) : rows((const bf16_t*)x, n, K, q, scale, st);
}

hipError_t launch_quantize_experts_fp8(const void* w, int dtype, int E, int K, int N, uint8_t* q, uint8_t* scale,
                                       hipStream_t st) {
    return dtype == MOE_F32 ? experts((const float*)w, E, K, N, q, scale, st)
                            : experts((const bf16_t*)w, E, K, N, q, scale, st);
}

}  // namespace moe
