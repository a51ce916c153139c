// The norms before and after a block, fused with the block's gate and residual scale, and
// their gradient (formulas: include/moe_ops.h).
//
//   v = z r(z) w_post    y = scale x + gate v    u = y r(y) w_next    r(t) = 1 / sqrt(mean t^2 + eps)
//
// Everything between the inputs and the rounded outputs is fp32, u from the unrounded y.  The
// gradient needs nothing but the inputs: with t = du w_next, and yh = y r(y), zh = z r(z),
//
//   g  = dy + r(y) (t - yh mean(t yh))                      the gradient of y
//   dx = scale g      p = g gate w_post      dz = r(z) (p - zh mean(p zh))
//   dw_next = sum du yh   dw_post = sum g gate zh   dgate = sum g w_post zh   (over rows, or columns)
//
// so a row costs one read of each input and one write of each output, with two (three)
// reductions over the row in between.  Memory bounds both kernels, so what counts is that loads
// are always on their way: the row stays in registers, 8 columns a thread, the next row's loads
// start before this row's reductions, and a thread's columns do not change, so that the
// parameters are read once and the sums over rows stay in registers until the end.  These are
// added up over workgroups by a second kernel, from partial sums in the caller's workspace, in a
// fixed order, without atomics.  Stores go through the caches, since the next operator reads them.
//
// Measured (bytes read and written once; a large copy moves 4.9 TB/s): forward 8192 x 4096 bf16
// 51 us (5.2 TB/s), 8192 x 7168 fp32 181 us (5.2), 32768 x 512 bf16 26 us (5.1); gradient
// 8192 x 7168 bf16 149 us (4.7), 8192 x 4096 fp32 173 us (4.7).  Rows of 264 to 1032 columns are
// slower: 4999 x 1032 fp32 43 us (2.9: 129 of a row's 192 threads have columns, and the second
// kernel is 5 us of it), bf16 28 (2.2: half the bytes on their way, one row ahead of 16 bytes a
// thread and input).
#include "common.h"
#include "launch.h"
#include "mm_launch.h"

namespace moe {

namespace {

template <typename T>
struct Chunk;                                 // 8 elements as they lie in memory
template <>
struct Chunk<bf16_t> {
    uint4 d;
    __device__ __forceinline__ void get(const bf16_t* p) { d = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void clear() { d = uint4{0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ void open(float (&v)[8]) const {
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) v[2 * q] = bf16lo_to_f32(w[q]), v[2 * q + 1] = bf16hi_to_f32(w[q]);
    }
    static __device__ __forceinline__ void put(bf16_t* p, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(p) = uint4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                             pack_bf16x2(v[6], v[7])};
    }
};
template <>
struct Chunk<float> {
    float4 a, b;
    __device__ __forceinline__ void get(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void open(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    static __device__ __forceinline__ void put(float* p, const float (&v)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};

// Sums over lanes, without LDS: over each 16 lanes (in all of them), and over a wavefront.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float sum16(float x) {
    x = dpp_add<0xB1, 0xf>(x);                // lane ^ 1
    x = dpp_add<0x4E, 0xf>(x);                // lane ^ 2
    x = dpp_add<0x141, 0xf>(x);               // mirrored in 8 lanes
    return dpp_add<0x140, 0xf>(x);            // mirrored in 16
}
__device__ __forceinline__ float wave_sum(float x) {
    x = sum16(x);
    x = dpp_add<0x142, 0xa>(x);               // lane 15 of rows 0 and 2 to the rows after them
    x = dpp_add<0x143, 0xc>(x);               // lane 31 to the upper half
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

// A row's threads: a wavefront (RPW = 4 rows in a workgroup of 256) or the workgroup (RPW = 1,
// as many wavefronts as the row needs), with C chunks of 8 columns each.
template <int RPW>
__device__ __forceinline__ int row_threads() { return RPW > 1 ? 64 : (int)blockDim.x; }
template <int RPW>
__device__ __forceinline__ int row_thread() { return RPW > 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x; }

// Sums of two numbers over the threads of a row.  `slot` alternates from call to call: a
// wavefront writes a slot again only after the barrier behind which all have read it.  red[.]
// of wavefronts that the workgroup lacks are zeros.
template <int RPW>
__device__ __forceinline__ float2 row_sum(float a, float b, float2 (*red)[16], int& slot) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (RPW == 1) {
        if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = float2{a, b};
        __syncthreads();
        const float2 r = red[slot][threadIdx.x & 15];
        a = sum16(r.x);
        b = sum16(r.y);
        slot ^= 1;
    }
    return float2{a, b};
}
__device__ __forceinline__ void clear_red(float2 (*red)[16]) {
    if (threadIdx.x < 32) red[threadIdx.x >> 4][threadIdx.x & 15] = float2{0.f, 0.f};      // at least a wavefront calls
    __syncthreads();
}

// This thread's columns of a vector of H parameters (1 where there is none).
template <int C>
__device__ __forceinline__ void get_params(const float* __restrict__ w, int P, int t, int H, float (&v)[C][8]) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c * P + t) * 8;
        Chunk<float> k;
        k.a = k.b = make_float4(1.f, 1.f, 1.f, 1.f);
        if (w && col < H) k.get(w + col);
        k.open(v[c]);
    }
}
template <int C, typename T>
__device__ __forceinline__ void get_row(const T* __restrict__ row, bool live, int P, int t, int H, Chunk<T> (&v)[C]) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c * P + t) * 8;
        v[c].clear();
        if (live && col < H) v[c].get(row + col);
    }
}

template <typename T, int RPW, int C>
__global__ __launch_bounds__(RPW > 1 ? 64 * RPW : 1024) void k_norm(NormArgs a) {
    __shared__ float2 red[2][16];
    if constexpr (RPW == 1) clear_red(red);
    int slot = 0;
    const int P = row_threads<RPW>(), t = row_thread<RPW>(), sub = RPW > 1 ? (int)(threadIdx.x >> 6) : 0, H = a.H;
    const long long first = (long long)blockIdx.x * RPW + sub, step = (long long)gridDim.x * RPW;
    const float over = 1.f / (float)H;
    const T *x = (const T*)a.x, *z = (const T*)a.z;
    float w1[C][8], gc[C][8], w2[C][8];
    get_params<C>(a.w_post, P, t, H, w1);
    get_params<C>(a.gate_kind == 1 ? a.gate : nullptr, P, t, H, gc);
    get_params<C>(a.w_next, P, t, H, w2);
    Chunk<T> xn[C], zn[C];
    get_row<C>(x + first * a.ldx, first < a.T, P, t, H, xn);
    get_row<C>(z + first * a.ldz, z && first < a.T, P, t, H, zn);
    // every row of threads runs the same number of rounds, so that the barriers match
    for (long long r0 = (long long)blockIdx.x * RPW; r0 < a.T; r0 += step) {
        const long long r = r0 + sub;
        const bool live = r < a.T;
        float y[C][8], v[C][8];
#pragma unroll
        for (int c = 0; c < C; ++c) xn[c].open(y[c]), zn[c].open(v[c]);
        const float gt = a.gate_kind == 2 && live ? a.gate[r] : 1.f;
        const bool more = r + step < a.T;
        get_row<C>(x + (r + step) * a.ldx, more, P, t, H, xn);
        get_row<C>(z + (r + step) * a.ldz, z && more, P, t, H, zn);
        if (z) {
            float rz = 1.f;
            if (a.w_post) {
                float s = 0.f;
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s = fmaf(v[c][j], v[c][j], s);
                rz = rsqrtf(row_sum<RPW>(s, 0.f, red, slot).x * over + a.eps);
            }
            const float f = rz * gt;
#pragma unroll
            for (int c = 0; c < C; ++c) {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[c][j] = fmaf(a.scale, y[c][j], v[c][j] * f * (w1[c][j] * gc[c][j]));
                const int col = (c * P + t) * 8;
                if (live && col < H) Chunk<T>::put((T*)a.y + r * H + col, y[c]);
            }
        }
        if (a.w_next) {
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(y[c][j], y[c][j], s);
            const float ry = rsqrtf(row_sum<RPW>(s, 0.f, red, slot).x * over + a.eps);
#pragma unroll
            for (int c = 0; c < C; ++c) {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[c][j] *= ry * w2[c][j];
                const int col = (c * P + t) * 8;
                if (live && col < H) Chunk<T>::put((T*)a.u + r * H + col, y[c]);
            }
        }
    }
}

// Rows side by side in a workgroup of `rpw` rows, P threads (whole wavefronts) each: the sums over
// rows then leave the workgroup once for all of them.  A thread has C chunks.
//   C = 1  parameters and all sums in registers, the next row's loads ahead.
//   C = 3  (rows above 8192, to 12288; 512 threads, for 256 registers each) two of the three sums over
//          rows live in LDS; parameters are read again for each row, from L2, all chunks' at once
//          and kept from one phase to the next.  4000 x 12288 bf16 183 us (3.2 TB/s), fp32 278
//          (4.2; measured beside the next three, 267); with the next row's loads ahead and parameters
//          read at each use 202 and 309, with both, which spills, 334; with C = 2 223 and 397.
//   C = 2  (longer rows; up to 1024 threads of 128 registers) as 3, but each parameter is read where
//          it is used.  3000 x 16384 bf16 218 us (2.7 TB/s), fp32 386 (3.1); C = 4 in 512 threads
//          spills: 229 to 383 and 435 to 458.
template <typename T, int C>
__global__ __launch_bounds__(C == 3 ? 512 : 1024) void k_norm_grad(NormGradArgs g, int P, int rpw) {
    constexpr bool HOLD = C == 1, KEEP = C == 3;        // parameters through all rows; through a row's phases
    const NormArgs& a = g.f;
    extern __shared__ float lds[];                      // sums of a row's columns: [P C 8], C > 1: twice
    __shared__ float2 red[2][16][16];                   // [slot][row][wavefront of the row]
    for (int i = threadIdx.x; i < 512; i += blockDim.x) red[i >> 8][(i >> 4) & 15][i & 15] = float2{0.f, 0.f};
    int slot = 0;
    const int H = a.H, wave = threadIdx.x >> 6, W = P >> 6;
    const int sub = __builtin_amdgcn_readfirstlane(wave / W), t = threadIdx.x - sub * P;
    const long long first = (long long)blockIdx.x * rpw + sub, step = (long long)gridDim.x * rpw;
    const float over = 1.f / (float)H;
    const T *x = (const T*)a.x, *z = (const T*)a.z, *dy = (const T*)g.dy, *du = (const T*)g.du;
    const bool need_z = z && (a.w_post || a.w_next || a.gate_kind), channel = a.gate_kind == 1;
    const float* gate_c = channel ? a.gate : nullptr;
    auto sum = [&](float p, float q) {
        p = wave_sum(p);
        q = wave_sum(q);
        if (W > 1) {
            if ((threadIdx.x & 63) == 0) red[slot][sub][wave - sub * W] = float2{p, q};
            __syncthreads();
            const float2 r = red[slot][sub][threadIdx.x & 15];
            p = sum16(r.x);
            q = sum16(r.y);
            slot ^= 1;
        }
        return float2{p, q};
    };
    float w1[HOLD ? C : 1][8], gc[HOLD ? C : 1][8], w2[HOLD ? C : 1][8];
    float s1[HOLD ? C : 1][8] = {}, sg[HOLD ? C : 1][8] = {}, s2[C][8] = {};
    if constexpr (HOLD) {
        get_params<C>(a.w_post, P, t, H, w1);
        get_params<C>(gate_c, P, t, H, gc);
        get_params<C>(a.w_next, P, t, H, w2);
    } else {
        for (int i = threadIdx.x; i < 2 * C * 8 * P; i += blockDim.x) lds[i] = 0.f;
    }
    __syncthreads();
    // chunk c's parameters
    auto param = [&](const float* w, const float (&held)[HOLD ? C : 1][8], int c, float (&v)[8]) {
        if constexpr (HOLD) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = held[c][j];
        } else {
            const int col = (c * P + t) * 8;
            Chunk<float> k;
            k.a = k.b = make_float4(1.f, 1.f, 1.f, 1.f);
            asm volatile("" : "+s"(w));                   // read where they are used, not kept through the rows
            if (w && col < H) k.get(w + col);
            k.open(v);
        }
    };
    Chunk<T> xn[C], zn[C], gn[C], un[C];
    auto start = [&](long long r) {
        const bool live = r < a.T;
        get_row<C>(x + r * a.ldx, live && a.w_next, P, t, H, xn);
        get_row<C>(z + r * a.ldz, live && need_z, P, t, H, zn);
        get_row<C>(dy + r * H, live && dy, P, t, H, gn);
        get_row<C>(du + r * H, live && a.w_next, P, t, H, un);
    };
    if constexpr (HOLD) start(first);
    // every row of threads runs the same number of rounds, so that the barriers match
    for (long long r0 = (long long)blockIdx.x * rpw; r0 < a.T; r0 += step) {
        const long long r = r0 + sub;
        const bool live = r < a.T;
        if constexpr (!HOLD) start(r);
        float xv[C][8], gv[C][8];
        Chunk<T> zc[C], uc[C];
#pragma unroll
        for (int c = 0; c < C; ++c) xn[c].open(xv[c]), gn[c].open(gv[c]), zc[c] = zn[c], uc[c] = un[c];
        const float gt = a.gate_kind == 2 && live ? a.gate[r] : 1.f;
        if constexpr (HOLD) start(r + step);
        float rz = 1.f;
        float k1[KEEP ? C : 1][8], k2[KEEP ? C : 1][8];
        auto keep_weights = [&] {                         // w_post and gate, before each phase that needs them
            if constexpr (KEEP)
#pragma unroll
                for (int c = 0; c < C; ++c) param(a.w_post, w1, c, k1[c]), param(gate_c, gc, c, k2[c]);
        };
        auto row_params = [&](int c, float (&p)[8], float (&q)[8]) {
            if constexpr (KEEP) {
#pragma unroll
                for (int j = 0; j < 8; ++j) p[j] = k1[c][j], q[j] = k2[c][j];
            } else {
                param(a.w_post, w1, c, p);
                param(gate_c, gc, c, q);
            }
        };
        auto row_weight = [&](int c, float (&v)[8]) {     // gate w_post
            float q[8];
            row_params(c, v, q);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= q[j];
        };
        if (a.w_next && z) keep_weights();
        if (a.w_post) {
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float zv[8];
                zc[c].open(zv);
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(zv[j], zv[j], s);
            }
            rz = rsqrtf(sum(s, 0.f).x * over + a.eps);
        }
        if (a.w_next) {
            float sy = 0.f, st = 0.f;
            if (z) {
                const float f = rz * gt;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float zv[8], w[8];
                    zc[c].open(zv);
                    row_weight(c, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) xv[c][j] = fmaf(a.scale, xv[c][j], zv[j] * f * w[j]);
                }
            }
            float k3[KEEP ? C : 1][8];
            if constexpr (KEEP)
#pragma unroll
                for (int c = 0; c < C; ++c) param(a.w_next, w2, c, k3[c]);
            auto next_weight = [&](int c, float (&v)[8]) {
                if constexpr (KEEP) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = k3[c][j];
                } else {
                    param(a.w_next, w2, c, v);
                }
            };
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float uv[8], w[8];
                uc[c].open(uv);
                next_weight(c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sy = fmaf(xv[c][j], xv[c][j], sy);
                    st = fmaf(uv[j] * w[j], xv[c][j], st);
                }
            }
            const float2 s = sum(sy, st);
            const float ry = rsqrtf(s.x * over + a.eps), k = ry * ry * (s.y * over);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float uv[8], w[8];
                uc[c].open(uv);
                next_weight(c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    gv[c][j] += ry * (uv[j] * w[j] - xv[c][j] * k);
                    s2[c][j] = fmaf(uv[j], xv[c][j] * ry, s2[c][j]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * P + t) * 8;
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = a.scale * gv[c][j];
            if (live && col < H) Chunk<T>::put((T*)g.dx + r * H + col, o);
        }
        if (z) {
            keep_weights();
            float k = 0.f;
            if (a.w_post || a.gate_kind == 2) {
                float s = 0.f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float zv[8], w[8];
                    zc[c].open(zv);
                    row_weight(c, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) s = fmaf(gv[c][j] * w[j], zv[j], s);
                }
                s = sum(s, 0.f).x;
                if (a.gate_kind == 2 && live && t == 0) g.dgate[r] = s * rz;
                if (a.w_post) k = s * rz * rz * over;
            }
            const float f = rz * gt;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int col = (c * P + t) * 8;
                float o[8], zv[8], p1[8], pg[8];
                zc[c].open(zv);
                row_params(c, pg, p1);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float q = gv[c][j] * (zv[j] * f);
                    o[j] = f * (gv[c][j] * (pg[j] * p1[j]) - zv[j] * k);
                    p1[j] *= q;
                    pg[j] *= q;
                }
                if (live && col < H) Chunk<T>::put((T*)g.dz + r * H + col, o);
                if constexpr (HOLD) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) s1[c][j] += p1[j], sg[c][j] += pg[j];
                } else {
                    // this thread's own places, 16 bytes a lane side by side
                    float4* l = reinterpret_cast<float4*>(lds) + (c * 4) * P + t;
                    auto add = [&](float4* at, const float* v) {
                        const float4 o4 = *at;
                        *at = make_float4(o4.x + v[0], o4.y + v[1], o4.z + v[2], o4.w + v[3]);
                    };
                    if (a.w_post) add(l, p1), add(l + P, p1 + 4);
                    if (channel) add(l + 2 * P, pg), add(l + 3 * P, pg + 4);
                }
            }
        }
    }
    // this workgroup's sums: [3][H] of the workspace, those of its rows added in order
    float* part = g.parts + (size_t)blockIdx.x * 3 * H;
    auto put = [&](int which, const float (&s)[8], int c) {
        const int col = (c * P + t) * 8;
        if (rpw == 1) {
            if (col < H) Chunk<float>::put(part + (size_t)which * H + col, s);
            return;
        }
        for (int k = 0; k < rpw; ++k) {
            __syncthreads();
            if (sub == k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float* p = lds + j * P + t;
                    *p = k ? *p + s[j] : s[j];
                }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 8 * P; i += blockDim.x)
            if (i % P * 8 + i / P < H) part[(size_t)which * H + i % P * 8 + i / P] = lds[i];
    };
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if constexpr (HOLD) {
            if (a.w_post) put(0, s1[c], c);
            if (channel) put(1, sg[c], c);
        } else {
            const float4* l = reinterpret_cast<const float4*>(lds) + (c * 4) * P + t;
            auto get = [&](int which) {
                const float4 p = l[2 * which * P], q = l[(2 * which + 1) * P];
                const float v[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
                put(which, v, c);
            };
            if (a.w_post) get(0);
            if (channel) get(1);
        }
        if (a.w_next) put(2, s2[c], c);
    }
}

// Adds the workgroups' sums: 64 columns per workgroup, its 16 wavefronts over the partial sums.
// What bounds it is the time of one load from L2 times the loads that wait for each other, hence
// eight in flight: 512 partial sums of 1032 to 7168 columns take 5 us (one in flight: 14).
__global__ __launch_bounds__(1024) void k_norm_reduce(const float* __restrict__ parts, int n, int H, float* d0, float* d1,
                                                      float* d2) {
    __shared__ float sums[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, which = blockIdx.y, col = blockIdx.x * 64 + lane;
    float* d = which == 0 ? d0 : which == 1 ? d1 : d2;
    if (!d) return;
    float s = 0.f;
    if (col < H) {
        const float* p = parts + (size_t)which * H + col;
        const size_t row = (size_t)3 * H;
        for (int i = wave; i < n; i += 16 * 8) {              // eight loads in flight
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = i + 16 * k < n ? p[(i + 16 * k) * row] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
        }
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && col < H) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += sums[i][lane];
        d[col] = s;
    }
}

// Threads of a row (forward): a chunk each up to 8192 columns, then two.
int row_threads_of(int H) { return ((H <= 8192 ? H / 8 : (H + 15) / 16) + 63) / 64 * 64; }
int grad_chunks_of(int H) { return H <= 8192 ? 1 : H <= 12288 ? 3 : 2; }      // (reasons: k_norm_grad)

constexpr int kMaxRow = 16384;

// Rows up to 512 columns: a wavefront each, four to a workgroup; longer ones a workgroup each.
template <typename T>
hipError_t go(const NormArgs& a, hipStream_t st) {
    const bool waves = a.H <= 512;
    const int NT = waves ? 256 : row_threads_of(a.H), rpw = waves ? 4 : 1;
    const long long want = (a.T + rpw - 1) / rpw, most = (long long)(1024 / NT < 1 ? 1 : 1024 / NT) * device_cu_count();
    const dim3 grid((unsigned)(want < most ? want : most));
    if (waves) hipLaunchKernelGGL((k_norm<T, 4, 1>), grid, dim3(NT), 0, st, a);
    else if (a.H <= 8192) hipLaunchKernelGGL((k_norm<T, 1, 1>), grid, dim3(NT), 0, st, a);
    else hipLaunchKernelGGL((k_norm<T, 1, 2>), grid, dim3(NT), 0, st, a);
    return hipGetLastError();
}

// The gradient has two workgroups of up to 512 threads for each of 256 CUs, or one: of up to 1024
// threads, or whose sums fill LDS.  With few rows, fewer rows side by side first.  Rows side by side
// leave one set of partial sums for all of them: 4999 x 1032 fp32 58 -> 43 us against one row a
// workgroup.
struct GradShape {
    int P, rpw, parts;
};
GradShape grad_shape(long long T, int H) {
    GradShape s;
    const int C = grad_chunks_of(H);
    s.P = (H / 8 + 64 * C - 1) / (64 * C) * 64;
    const bool two = C == 1 && s.P <= 512;
    const int most = two ? 512 : 256;
    const long long share = (T + most - 1) / most, fit = two ? 512 / s.P : 1;
    s.rpw = (int)(share < 1 ? 1 : share < fit ? share : fit);
    const long long want = (T + s.rpw - 1) / s.rpw;
    s.parts = (int)(want < most ? want : most);
    return s;
}

template <typename T>
hipError_t go_grad(const NormGradArgs& g, hipStream_t st) {
    const GradShape s = grad_shape(g.f.T, g.f.H);
    const dim3 grid((unsigned)s.parts), threads((unsigned)(s.P * s.rpw));
    if (g.f.H <= 8192) {
        hipLaunchKernelGGL((k_norm_grad<T, 1>), grid, threads, (size_t)s.P * 8 * 4, st, g, s.P, s.rpw);
    } else {
        const int C = grad_chunks_of(g.f.H);
        const size_t lds = (size_t)s.P * C * 8 * 4 * 2;
        const hipError_t e = C == 3 ? allow_lds<k_norm_grad<T, 3>>(2 * 12288 * sizeof(float))
                                    : allow_lds<k_norm_grad<T, 2>>(2 * kMaxRow * sizeof(float));
        if (e != hipSuccess) return e;
        if (C == 3) hipLaunchKernelGGL((k_norm_grad<T, 3>), grid, threads, lds, st, g, s.P, s.rpw);
        else hipLaunchKernelGGL((k_norm_grad<T, 2>), grid, threads, lds, st, g, s.P, s.rpw);
    }
    return hipGetLastError();
}

}  // namespace

int norm_grad_parts(long long T, int H) { return grad_shape(T, H).parts; }

hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t st) {
    return dtype == MOE_F32 ? go<float>(a, st) : go<bf16_t>(a, st);
}

hipError_t launch_norm_grad(const NormGradArgs& g, int dtype, hipStream_t st) {
    if (g.f.T > 0) {
        const hipError_t e = dtype == MOE_F32 ? go_grad<float>(g, st) : go_grad<bf16_t>(g, st);
        if (e != hipSuccess) return e;
    }
    float* dgate = g.f.gate_kind == 1 ? g.dgate : nullptr;
    if (!g.dw_post && !dgate && !g.dw_next) return hipSuccess;
    hipLaunchKernelGGL(k_norm_reduce, dim3((unsigned)((g.f.H + 63) / 64), 3), dim3(1024), 0, st, g.parts,
                       norm_grad_parts(g.f.T, g.f.H), g.f.H, g.dw_post, dgate, g.dw_next);
    return hipGetLastError();
}

}  // namespace moe
