// Counter-based dropout, alone and fused with the experts' gated activation, and its
// gradient.
//
//   keep(i) = u(i) >= t,  t = round(65536 p),  c = 65536 / (65536 - t)
//   dropout y = keep ? c x : 0
//   gated   h = keep ? c SiLU(a) b : 0           (b = 1 without an up projection)
//   gradient, with d = keep ? c dh : 0 and s = 1 / (1 + exp(-a)):
//           da = d b s (1 + a (1 - s)),  db = d a s
//
// u(i) is a 16-bit number of a counter-based generator, Philox4x32-10 (Salmon, Moraes,
// Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011): element i of the
// row-major tensor takes lane i mod 8 of block i div 8, a block being four 32-bit words
// read as eight 16-bit numbers, low half first.  So the mask is a function of (seed,
// step, i) and is never stored: the gradient computes it again.
//
// Sixteen bits an element, so that one block serves the eight bf16 values of a 16-byte
// access.  p is then a multiple of 2^-16; c is made from the rounded p, which keeps the
// expectation exact.
//
// A dropped element is selected away, not multiplied by zero: an infinity or a NaN under
// the mask does not reach the result.
//
// Memory bounds all of them: eight elements a thread, one pass, the generator's ten rounds
// (some 60 integer instructions a block) under the loads.  8192 x 14336 bf16, h from a packed
// pair: 121 us, 5.8 TB/s; its kind of gradient over 65536 x 2048: 232 us, 5.8 TB/s; 256 x
// 4096, plain: 3.0 us, the launch.
#include "common.h"
#include "launch.h"
#include "mm_launch.h"

namespace moe {

namespace {

struct Philox {
    uint32_t w[4];
    // 16-bit number of lane j (0..7), low half first
    __device__ __forceinline__ uint32_t u16(int j) const { return (w[j >> 1] >> (16 * (j & 1))) & 0xffffu; }
};

__device__ __forceinline__ Philox philox(uint64_t block, uint64_t step, uint64_t seed) {
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)step, c3 = (uint32_t)(step >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Philox{{c0, c1, c2, c3}};
}

// eight consecutive elements, in fp32
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        const uint4 d = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) v[2 * q] = bf16lo_to_f32(w[q]), v[2 * q + 1] = bf16hi_to_f32(w[q]);
    } else {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p) = uint4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                             pack_bf16x2(v[6], v[7])};
    } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}
__device__ __forceinline__ float get1(const float* p) { return *p; }
__device__ __forceinline__ float get1(const bf16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ void put1(bf16_t* p, float v) { *p = f32_to_bf16(v); }

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

// The step of this launch: the caller's, plus a device word where one is given (a captured
// launch then draws a new mask at each replay).
__device__ __forceinline__ uint64_t step_of(const DropArgs& d) { return d.step + (d.step_ptr ? *d.step_ptr : 0); }

template <bool DROP>
__device__ __forceinline__ Philox draw8(uint64_t block, const DropArgs& d) {
    if constexpr (DROP) return philox(block, step_of(d), d.seed);
    else return Philox{};
}
template <bool DROP>
__device__ __forceinline__ bool keep(const Philox& r, int j, const DropArgs& d) {
    return !DROP || r.u16(j) >= d.thr;
}

template <typename T, bool DROP>
__global__ __launch_bounds__(256) void k_dropout(const T* x, T* y, long long n, DropArgs d) {
    const long long blk = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long i = blk * 8;
    if (i >= n) return;
    const Philox r = draw8<DROP>(blk, d);
    if (i + 8 <= n) {
        float v[8];
        load8(x + i, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = keep<DROP>(r, j, d) ? v[j] * d.scale : 0.f;
        store8(y + i, v);
    } else {
        for (int j = 0; j < 8; ++j)
            if (i + j < n) put1(y + i + j, keep<DROP>(r, j, d) ? get1(x + i + j) * d.scale : 0.f);
    }
}

template <typename T, bool GATE, bool DROP>
__global__ __launch_bounds__(256) void k_gated_act(const T* __restrict__ a, long long lda, const T* __restrict__ b,
                                                   long long ldb, T* __restrict__ h, long long blocks, int f8,
                                                   DropArgs d) {
    const long long blk = (long long)blockIdx.x * 256 + threadIdx.x;
    if (blk >= blocks) return;
    const long long row = blk / f8;
    const int col = (int)(blk - row * f8) * 8;
    const Philox r = draw8<DROP>(blk, d);
    float av[8], bv[8];
    load8(a + row * lda + col, av);
    if constexpr (GATE) load8(b + row * ldb + col, bv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float s, ns;
        sigmoid<sizeof(T) == 2>(av[j], s, ns);
        float v = av[j] * s;
        if constexpr (GATE) v *= bv[j];
        av[j] = keep<DROP>(r, j, d) ? v * d.scale : 0.f;
    }
    store8(h + blk * 8, av);
}

template <typename T, bool GATE, bool DROP>
__global__ __launch_bounds__(256) void k_gated_act_grad(const T* __restrict__ dh, const T* __restrict__ a,
                                                        long long lda, const T* __restrict__ b, long long ldb,
                                                        T* __restrict__ da, long long ldda, T* __restrict__ db,
                                                        long long lddb, long long blocks, int f8, DropArgs d) {
    const long long blk = (long long)blockIdx.x * 256 + threadIdx.x;
    if (blk >= blocks) return;
    const long long row = blk / f8;
    const int col = (int)(blk - row * f8) * 8;
    const Philox r = draw8<DROP>(blk, d);
    float av[8], bv[8], g[8];
    load8(a + row * lda + col, av);
    if constexpr (GATE) load8(b + row * ldb + col, bv);
    load8(dh + blk * 8, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float s, ns;
        sigmoid<sizeof(T) == 2>(av[j], s, ns);
        const bool k = keep<DROP>(r, j, d);
        const float gj = g[j] * d.scale;
        float va = gj * (s * (1.f + av[j] * ns));
        if constexpr (GATE) va *= bv[j], bv[j] = k ? gj * (av[j] * s) : 0.f;
        av[j] = k ? va : 0.f;
    }
    store8(da + row * ldda + col, av);
    if constexpr (GATE) store8(db + row * lddb + col, bv);
}

unsigned grid_of(long long blocks) { return (unsigned)((blocks + 255) / 256); }

template <typename T, bool DROP>
void act(const void* a, long long lda, const void* b, long long ldb, void* h, long long rows, int F, const DropArgs& d,
         hipStream_t st) {
    const long long n = rows * (F / 8);
    if (b)
        hipLaunchKernelGGL((k_gated_act<T, true, DROP>), dim3(grid_of(n)), dim3(256), 0, st, (const T*)a, lda,
                           (const T*)b, ldb, (T*)h, n, F / 8, d);
    else
        hipLaunchKernelGGL((k_gated_act<T, false, DROP>), dim3(grid_of(n)), dim3(256), 0, st, (const T*)a, lda,
                           (const T*)b, ldb, (T*)h, n, F / 8, d);
}

template <typename T, bool DROP>
void act_grad(const void* dh, const void* a, long long lda, const void* b, long long ldb, void* da, long long ldda,
              void* db, long long lddb, long long rows, int F, const DropArgs& d, hipStream_t st) {
    const long long n = rows * (F / 8);
    if (b)
        hipLaunchKernelGGL((k_gated_act_grad<T, true, DROP>), dim3(grid_of(n)), dim3(256), 0, st, (const T*)dh,
                           (const T*)a, lda, (const T*)b, ldb, (T*)da, ldda, (T*)db, lddb, n, F / 8, d);
    else
        hipLaunchKernelGGL((k_gated_act_grad<T, false, DROP>), dim3(grid_of(n)), dim3(256), 0, st, (const T*)dh,
                           (const T*)a, lda, (const T*)b, ldb, (T*)da, ldda, (T*)db, lddb, n, F / 8, d);
}

}  // namespace

hipError_t launch_dropout(const void* x, void* y, int dtype, long long n, const DropArgs& d, hipStream_t st) {
    const dim3 g(grid_of((n + 7) / 8)), t(256);
    if (dtype == MOE_BF16) {
        if (d.thr) hipLaunchKernelGGL((k_dropout<bf16_t, true>), g, t, 0, st, (const bf16_t*)x, (bf16_t*)y, n, d);
        else hipLaunchKernelGGL((k_dropout<bf16_t, false>), g, t, 0, st, (const bf16_t*)x, (bf16_t*)y, n, d);
    } else {
        if (d.thr) hipLaunchKernelGGL((k_dropout<float, true>), g, t, 0, st, (const float*)x, (float*)y, n, d);
        else hipLaunchKernelGGL((k_dropout<float, false>), g, t, 0, st, (const float*)x, (float*)y, n, d);
    }
    return hipGetLastError();
}

hipError_t launch_gated_act(const void* a, long long lda, const void* b, long long ldb, void* h, int dtype,
                            long long rows, int F, const DropArgs& d, hipStream_t st) {
    if (dtype == MOE_BF16) d.thr ? act<bf16_t, true>(a, lda, b, ldb, h, rows, F, d, st)
                                 : act<bf16_t, false>(a, lda, b, ldb, h, rows, F, d, st);
    else d.thr ? act<float, true>(a, lda, b, ldb, h, rows, F, d, st)
               : act<float, false>(a, lda, b, ldb, h, rows, F, d, st);
    return hipGetLastError();
}

hipError_t launch_gated_act_grad(const void* dh, const void* a, long long lda, const void* b, long long ldb, void* da,
                                 long long ldda, void* db, long long lddb, int dtype, long long rows, int F,
                                 const DropArgs& d, hipStream_t st) {
    if (dtype == MOE_BF16) d.thr ? act_grad<bf16_t, true>(dh, a, lda, b, ldb, da, ldda, db, lddb, rows, F, d, st)
                                 : act_grad<bf16_t, false>(dh, a, lda, b, ldb, da, ldda, db, lddb, rows, F, d, st);
    else d.thr ? act_grad<float, true>(dh, a, lda, b, ldb, da, ldda, db, lddb, rows, F, d, st)
               : act_grad<float, false>(dh, a, lda, b, ldb, da, ldda, db, lddb, rows, F, d, st);
    return hipGetLastError();
}

}  // namespace moe
