// Helpers of the grouped products (mm.hip, mm_stream.hip, mm_mid.hip, mm_thin.hip): row groups and row tiles.
#pragma once

#include "common.h"

namespace moe {

// Rows of group e as the offsets give them, clamped into [0, rows] so that no offset
// array, whatever it holds, leads outside the row buffers.
__device__ __forceinline__ void group_rows(const int32_t* __restrict__ offsets, int e, int rows, int& r0, int& r1) {
    r0 = min(max(offsets[e], 0), rows);
    r1 = min(max(offsets[e + 1], r0), rows);
}

// The groups as every workgroup keeps them in LDS: their rows, and the row tiles before each
// (pre[e]; pre[E] = all).  Computed from the offsets by every workgroup (at most 256 groups,
// four per lane of one wavefront), which saves the launch and the workspace of a tile list.
struct Groups {
    int r0[256], r1[256], pre[257];
};

// Fills `g` for tiles of BM rows.  Call with all threads.
__device__ __forceinline__ void load_groups(const int32_t* __restrict__ offsets, int E, int rows, int BM, Groups& g) {
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int n[4], sum = 0;
        // groups 4 lane .. 4 lane + 3: five offsets, the loads all in flight together
        int off[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) off[i] = offsets[min(4 * lane + i, E)];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 4 * lane + i, r0 = min(max(off[i], 0), rows), r1 = min(max(off[i + 1], r0), rows);
            if (e < E) {
                g.r0[e] = r0;
                g.r1[e] = r1;
            }
            n[i] = e < E ? (r1 - r0 + BM - 1) / BM : 0;
            sum += n[i];
        }
        int incl = sum;
        if (E > 3) {                                  // else lane 0 holds them all
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int v = __shfl_up(incl, o);
                if (lane >= o) incl += v;
            }
        }
        int p = incl - sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (4 * lane + i <= E) g.pre[4 * lane + i] = p;
            p += n[i];
        }
        if (lane == 63 && E == 256) g.pre[256] = incl;
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
