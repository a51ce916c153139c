// Host-side launchers of the training and 8-bit operators (moe_ops.h).  Each enqueues on
// `st` and returns the launch status; arguments were checked by the C ABI layer.
#pragma once

#include <atomic>

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct MmArgs {
    const void *a, *b;            // operands (see the kinds in mm_tile.h)
    void* c;
    const int32_t* offsets;
    const float *xs, *ws;         // int8: row and column scales
    int rows, E, K, N;
    int zero_rest;
};

// kind: 0 y = x W, 1 dx = dy W^T, 2 dW = x^T dy, 3 int8; in the form that suits the sizes
hipError_t launch_mm(int kind, int dtype, int out_dtype, const MmArgs& a, hipStream_t st);
// whether a launch can hold the call's workgroups
bool mm_fits(int kind, int dtype, const MmArgs& a);
// the form it takes on a GPU of `cus` compute units, as moe_grouped_mm_form names it (mm_fits)
const char* mm_form(int kind, int dtype, const MmArgs& a, int cus);
// the forms: 256 x 256 tiles (bf16, int8); tiles of 64 or 128 (fp32: 64); 16 or 32 rows with the
// contraction split over 8 or 4 wavefronts (kind 2: 32 rows)
bool mm_streams(const MmArgs& a);         // whether large weight gradients go in a stream of tiles
hipError_t launch_mm_stream(int out_dtype, const MmArgs& a, hipStream_t st);              // kind 2 of large
hipError_t launch_mm_large(int kind, int out_dtype, const MmArgs& a, hipStream_t st);
hipError_t launch_mm_mid(int tile, int kind, int dtype, int out_dtype, const MmArgs& a, hipStream_t st);
hipError_t launch_mm_thin(int rows, int kind, int dtype, int out_dtype, const MmArgs& a, hipStream_t st);

hipError_t launch_quantize_rows(const void* x, int dtype, long long rows, int K, int8_t* q, float* scale,
                                hipStream_t st);
hipError_t launch_quantize_experts(const void* w, int dtype, int E, int K, int N, int8_t* q, float* scale,
                                   hipStream_t st);

// Lets kernel KERN use `bytes` of dynamic LDS on the current device (asked of the runtime once
// per kernel and device).
template <auto KERN>
hipError_t allow_lds(size_t bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    e = hipFuncSetAttribute((const void*)KERN, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

struct DropArgs {
    uint32_t thr;                 // elements whose 16-bit number is below are dropped (0..65536)
    float scale;
    uint64_t seed, step;
    const uint64_t* step_ptr;     // NULL, or a device word added to step
};
hipError_t launch_dropout(const void* x, void* y, int dtype, long long n, const DropArgs& d, hipStream_t st);
hipError_t launch_gated_act(const void* a, long long lda, const void* b, long long ldb, void* h, int dtype,
                            long long rows, int F, const DropArgs& d, hipStream_t st);
hipError_t launch_gated_act_grad(const void* dh, const void* a, long long lda, const void* b, long long ldb, void* da,
                                 long long ldda, void* db, long long lddb, int dtype, long long rows, int F,
                                 const DropArgs& d, hipStream_t st);

hipError_t launch_combine_grad(const void* dout, const void* y_perm, const int32_t* row_of_pair, const float* w,
                               void* dy_perm, float* dw, long long T, int k, int H, int dtype, long long rows,
                               hipStream_t st);

}  // namespace moe
