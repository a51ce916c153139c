// Helpers of the grouped products (mm.hip, mm_f32.hip): row groups and row tiles.
#pragma once

#include "common.h"

namespace moe {

// Rows of group e as the offsets give them, clamped into [0, rows] so that no offset
// array, whatever it holds, leads outside the row buffers.
__device__ __forceinline__ void group_rows(const int32_t* __restrict__ offsets, int e, int rows, int& r0, int& r1) {
    r0 = min(max(offsets[e], 0), rows);
    r1 = min(max(offsets[e + 1], r0), rows);
}

// Row tiles of all groups, without a tile list in memory: pre[e] = tiles of the groups
// before e (BM rows each), pre[E] = all.  Every workgroup computes it from the offsets (at
// most 256 groups, four per lane of one wavefront), which saves the launch and the
// workspace of a list.  Call with all threads; `pre` holds 257 ints of LDS.
__device__ __forceinline__ void build_row_tiles(const int32_t* __restrict__ offsets, int E, int rows, int BM,
                                                int* pre) {
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int n[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 4 * lane + i;
            int r0 = 0, r1 = 0;
            if (e < E) group_rows(offsets, e, rows, r0, r1);
            n[i] = (r1 - r0 + BM - 1) / BM;
            sum += n[i];
        }
        int incl = sum;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(incl, off);
            if (lane >= off) incl += v;
        }
        int p = incl - sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (4 * lane + i <= E) pre[4 * lane + i] = p;
            p += n[i];
        }
        if (lane == 63 && E == 256) pre[256] = incl;
    }
    __syncthreads();
}

// The group of row tile t (t < pre[E]), found by all lanes of a wavefront together: the
// number of groups whose first tile is at or before t, less one.  (Groups without rows
// share their first tile with the next group that has some; the last of them is taken.)
__device__ __forceinline__ int group_of_tile(const int* pre, int E, int t) {
    const int lane = threadIdx.x & 63;
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = lane + 64 * i;
        cnt += __popcll(__ballot(e < E && pre[e] <= t));
    }
    return cnt - 1;
}

// Zeros to the rows of out [rows, row_bytes] that lie in no group: before offsets[0] and
// from offsets[E] on.  row_bytes is a multiple of 16.  Shared out over the whole grid.
__device__ __forceinline__ void zero_rest(const int32_t* __restrict__ offsets, int E, int rows, void* out,
                                          long long row_bytes, long long block, long long nblocks) {
    const int lo = min(max(offsets[0], 0), rows), hi = min(max(offsets[E], lo), rows);
    const long long cpr = row_bytes / 16;
    const long long head = lo * cpr, n = head + (rows - hi) * cpr;
    for (long long i = block * blockDim.x + threadIdx.x; i < n; i += nblocks * blockDim.x) {
        const long long c = i < head ? i : hi * cpr + (i - head);
        reinterpret_cast<uint4*>(out)[c] = uint4{0u, 0u, 0u, 0u};
    }
}

}  // namespace moe
