// Grouped products, plain form of the kernels: one 64 x 64 output tile per workgroup.
//   kind 0  y[r, n]     = sum_k x[r, k] w[e, k, n]     (rows of group e)
//   kind 1  dx[r, k]    = sum_n dy[r, n] w[e, k, n]
//   kind 2  dw[e, k, n] = sum_r x[r, k] dy[r, n]       (zeros for a group without rows)
//   int8    y[r, n]     = (sum_k xq[r, k] wq[e, n, k]) * xs[r] * ws[e, n]
#include "common.h"
#include "launch.h"
#include "mm_common.h"
#include "mm_launch.h"

namespace moe {

namespace {

__device__ __forceinline__ float to_acc(float v) { return v; }
__device__ __forceinline__ float to_acc(bf16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ int to_acc(int8_t v) { return v; }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16_t* p, float v) { *p = f32_to_bf16(v); }

template <int KIND, typename TI, typename TO, typename ACC>
__global__ __launch_bounds__(256) void k_mm_simple(MmArgs a) {
    constexpr int TM = 64, TN = 64, TK = 16;
    __shared__ ACC sA[TK][TM + 4], sB[TK][TN + 4];
    __shared__ int pre[257];
    const int tid = threadIdx.x, tr = tid >> 4, tc = tid & 15;
    int e, i0, i1, j0 = blockIdx.y * TN, c1;            // output rows [i0, i1), first column, contraction length
    const int J = KIND == 1 ? a.K : a.N;
    const TI *A, *B;
    long long sai, sac, sbc, sbj;                       // element strides of A (row, contraction), B (contraction, column)
    TO* C;
    if constexpr (KIND == 2) {
        const int kt = (a.K + TM - 1) / TM;
        e = blockIdx.x / kt;
        int r0, r1;
        group_rows(a.offsets, e, a.rows, r0, r1);
        i0 = (blockIdx.x % kt) * TM;
        i1 = min(i0 + TM, a.K);
        c1 = r1 - r0;
        A = (const TI*)a.a + (long long)r0 * a.K, sai = 1, sac = a.K;
        B = (const TI*)a.b + (long long)r0 * a.N, sbc = a.N, sbj = 1;
        C = (TO*)a.c + (long long)e * a.K * a.N;
    } else {
        build_row_tiles(a.offsets, a.E, a.rows, TM, pre);
        if (a.zero_rest)
            zero_rest(a.offsets, a.E, a.rows, a.c, (long long)J * sizeof(TO),
                      blockIdx.x * (long long)gridDim.y + blockIdx.y, (long long)gridDim.x * gridDim.y);
        if ((int)blockIdx.x >= pre[a.E]) return;
        e = group_of_tile(pre, a.E, blockIdx.x);
        int r0, r1;
        group_rows(a.offsets, e, a.rows, r0, r1);
        i0 = r0 + ((int)blockIdx.x - pre[e]) * TM;
        i1 = min(i0 + TM, r1);
        c1 = KIND == 1 ? a.N : a.K;
        A = (const TI*)a.a, sai = c1, sac = 1;
        B = (const TI*)a.b + (long long)e * a.K * a.N;
        if constexpr (KIND == 0) sbc = a.N, sbj = 1;
        else if constexpr (KIND == 1) sbc = 1, sbj = a.N;
        else sbc = 1, sbj = a.K;                        // int8: wq [E, N, K]
        C = (TO*)a.c;
    }
    ACC acc[4][4] = {};
    for (int c0 = 0; c0 < c1; c0 += TK) {
        for (int t = tid; t < TK * TM; t += 256) {
            const int c = sac == 1 ? t % TK : t / TM, i = sac == 1 ? t / TK : t % TM;
            sA[c][i] = (c0 + c < c1 && i0 + i < i1) ? to_acc(A[(i0 + i) * sai + (c0 + c) * sac]) : (ACC)0;
        }
        for (int t = tid; t < TK * TN; t += 256) {
            const int c = sbc == 1 ? t % TK : t / TN, j = sbc == 1 ? t / TK : t % TN;
            sB[c][j] = (c0 + c < c1 && j0 + j < J) ? to_acc(B[(c0 + c) * sbc + (j0 + j) * sbj]) : (ACC)0;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < TK; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += sA[c][tr * 4 + i] * sB[c][tc * 4 + j];
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = i0 + tr * 4 + i, n = j0 + tc * 4 + j;
            if (r >= i1 || n >= J) continue;
            float v = (float)acc[i][j];
            if constexpr (KIND == 3) v = v * a.xs[r] * a.ws[(long long)e * a.N + n];
            put(C + (long long)r * J + n, v);
        }
}

template <int KIND, typename TI, typename TO, typename ACC>
hipError_t go(const MmArgs& a, hipStream_t st) {
    const int J = KIND == 1 ? a.K : a.N;
    const long long nx = KIND == 2 ? (long long)a.E * ((a.K + 63) / 64)
                                   : ((long long)a.rows + 63) / 64 + (a.rows < a.E ? a.rows : a.E);
    hipLaunchKernelGGL((k_mm_simple<KIND, TI, TO, ACC>), dim3((unsigned)nx, (J + 63) / 64), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mm_simple(int kind, int dtype, int out_dtype, const MmArgs& a, hipStream_t st) {
    if (kind == 3) return out_dtype == MOE_BF16 ? go<3, int8_t, bf16_t, int>(a, st) : go<3, int8_t, float, int>(a, st);
    if (dtype == MOE_F32)
        return kind == 0 ? go<0, float, float, float>(a, st)
               : kind == 1 ? go<1, float, float, float>(a, st) : go<2, float, float, float>(a, st);
    if (kind == 2)
        return out_dtype == MOE_BF16 ? go<2, bf16_t, bf16_t, float>(a, st) : go<2, bf16_t, float, float>(a, st);
    return kind == 0 ? go<0, bf16_t, bf16_t, float>(a, st) : go<1, bf16_t, bf16_t, float>(a, st);
}

}  // namespace moe
