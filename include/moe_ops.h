/*
 * moe_ops.h -- operators beside the layer forward of moe.h (MI355X, gfx950): what training
 * the layer and serving it with 8-bit experts need.
 *
 *   grouped products   y = x W_e over ragged row groups, and both gradients
 *   8-bit integers     per-token and per-channel quantisation, and the grouped product
 *   dropout            counter-based, its mask never stored; alone or with the experts'
 *                      gated activation, and the gradient of that
 *   combine's gradient
 *
 * Conventions are those of moe.h: device pointers, 16-byte aligned; dense row-major arrays
 * unless a row stride is given; calls only enqueue on `stream`; nothing is allocated or
 * kept; arguments are checked on the host before anything is enqueued (moe_status, the
 * detail in moe_last_error()).  None of these calls needs a workspace, so any number of
 * them may run at the same time, captured or not, on buffers of their own.  Outputs must
 * not overlap inputs, except that moe_dropout may work in place.
 *
 * Results are deterministic: every output is written by one workgroup, sums run in a fixed
 * order, and there are no atomics on results.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A grouped product.  `rows` rows lie in E consecutive groups: group e holds the rows
 * [offsets[e], offsets[e+1]) (offsets [E+1] int32 on the device, as moe_permute writes
 * them).  Group sizes are arbitrary, zero among them; rows before offsets[0] and from
 * offsets[E] on belong to no group.  Offsets must not decrease; whatever they hold,
 * nothing outside the buffers is read or written.
 * Limits: 0 <= rows < 2^30; 1 <= E <= 256; K and N multiples of 8, at most 2^20; the output's
 * tiles within one launch (2^23 of 256 x 256, fp32 2^24 of 64 x 64; MOE_ERR_UNSUPPORTED
 * beyond).  moe_grouped_mm_int8: K a multiple of 16, at most 131056, so that no 32-bit sum
 * can overflow. */
typedef struct {
    int64_t  rows;
    int32_t  E, K, N;
    int32_t  dtype;      /* MOE_F32 or MOE_BF16: x, w, dy (see moe_grouped_mm_int8 for its own) */
    int32_t  out_dtype;  /* type of the output: dtype; moe_grouped_mm_dw on bf16 also MOE_F32 */
    uint32_t flags;      /* 0 or MOE_MM_ZERO_REST */
} moe_mm_shape;

/* Rows of y / dx that lie in no group are written as zeros.  Without it they are left as
 * they were. */
#define MOE_MM_ZERO_REST 0x1u

/* y[r] = x[r] W_e for the rows r of every group e.
 *   x [rows, K], w [E, K, N], y [rows, N] out.  Sums in fp32, one rounding.
 *   rows == 0 returns MOE_OK and enqueues nothing (row arrays may then be NULL). */
moe_status moe_grouped_mm(const moe_mm_shape* shape, const void* x, const void* w, const int32_t* offsets,
                          void* y, hipStream_t stream);

/* The gradient of moe_grouped_mm by x: dx[r] = dy[r] W_e^T.
 *   dy [rows, N], w [E, K, N], dx [rows, K] out. */
moe_status moe_grouped_mm_dx(const moe_mm_shape* shape, const void* dy, const void* w, const int32_t* offsets,
                             void* dx, hipStream_t stream);

/* The gradient of moe_grouped_mm by w: dw[e] = sum over the rows r of group e of
 * x[r]^T dy[r]; zeros for a group without rows.
 *   x [rows, K], dy [rows, N], dw [E, K, N] out, fully overwritten (also when rows == 0). */
moe_status moe_grouped_mm_dw(const moe_mm_shape* shape, const void* x, const void* dy, const int32_t* offsets,
                             void* dw, hipStream_t stream);

/* The kernel form that a product of these sizes takes on a GPU of `cus` compute units (0: of the
 * current device): "256x256", "256x256 stream" (weight gradients), "128x128", "64x64", "32x64
 * thin" or "16x64 thin".  Forms differ in speed and in the order of their sums.  For tests and
 * for reading traces; enqueues nothing, and with cus > 0 needs no GPU.  NULL where the product
 * would be refused (the reason in moe_last_error()). */
typedef enum { MOE_MM_Y = 0, MOE_MM_DX = 1, MOE_MM_DW = 2, MOE_MM_INT8 = 3 } moe_mm_product;
const char* moe_grouped_mm_form(const moe_mm_shape* shape, int32_t product, int32_t cus);

/* 8-bit rows: scale[r] = max_k |x[r, k]| / 127 in fp32, q[r, k] = x[r, k] / scale[r] to the
 * nearest integer (ties to even), in [-127, 127].  A row of zeros has scale 0 and q 0; a
 * row that holds an infinity or a NaN has scale NaN and q 0.
 *   x [rows, K] dtype, q [rows, K] int8 out, scale [rows] fp32 out; K a multiple of 8;
 *   rows < 2^24. */
moe_status moe_quantize_rows(int32_t dtype, int64_t rows, int32_t K, const void* x, int8_t* q, float* scale,
                             hipStream_t stream);

/* 8-bit experts, made once: w [E, K, N] dtype -> q [E, N, K] int8 (contraction contiguous),
 * scale [E, N] fp32, each output channel of each expert quantised over K as a row above.
 *   E <= 256; K a multiple of 16, at most 131056, N of 8, at most 2^20. */
moe_status moe_quantize_experts(int32_t dtype, int32_t E, int32_t K, int32_t N, const void* w, int8_t* q,
                                float* scale, hipStream_t stream);

/* y[r, n] = (sum_k xq[r, k] wq[e, n, k]) * x_scale[r] * w_scale[e, n]: the sum exact in
 * int32, converted to fp32, times the row's and then the channel's scale, one rounding to
 * out_dtype (MOE_BF16 or MOE_F32; shape->dtype is ignored).
 *   xq [rows, K] int8, x_scale [rows] fp32, wq [E, N, K] int8, w_scale [E, N] fp32,
 *   y [rows, N] out. */
moe_status moe_grouped_mm_int8(const moe_mm_shape* shape, const int8_t* xq, const float* x_scale,
                               const int8_t* wq, const float* w_scale, const int32_t* offsets, void* y,
                               hipStream_t stream);

/* Counter-based dropout.  t = round(65536 p), c = 65536 / (65536 - t); element i of the
 * row-major tensor is kept where u(i) >= t and then multiplied by c, else it is 0 (also
 * where it was an infinity or a NaN).  u(i) is lane i mod 8 of block i div 8 of
 * Philox4x32-10, a block being its four output words read as eight 16-bit numbers, low
 * half first; counter (block low, block high, step low, step high), key (seed low, seed
 * high).  The same (seed, step) gives the same mask, in the gradient too; use another step
 * for every tensor and training step.  step_device, if not NULL, is a device word (8-byte
 * aligned) added to step when the kernel runs, so that a captured launch can draw another
 * mask at every replay.  0 <= p <= 1. */
typedef struct {
    double   p;
    uint64_t seed, step;
    const uint64_t* step_device;
} moe_dropout_spec;

/* y[i] = keep(i) ? c x[i] : 0 for n elements of dtype; y may be x.  Also its own gradient:
 * dx = dropout(dy) with the same spec.  n < 2^34. */
moe_status moe_dropout(int32_t dtype, int64_t n, const moe_dropout_spec* spec, const void* x, void* y,
                       hipStream_t stream);

/* h = keep ? c SiLU(a) b : 0, the experts' activation ([Principles §3.1], [FourStage §2])
 * with dropout; b NULL: h = keep ? c SiLU(a) : 0.
 *   a, b [rows, F] dtype with lda / ldb elements from one row to the next (multiples of 8,
 *   at least F: the halves of a packed [rows, 2 F] tensor are such), h [rows, F] dense.
 *   Element (r, f) draws the number of index r F + f.  F a multiple of 8, rows F < 2^34. */
moe_status moe_gated_act(int32_t dtype, int64_t rows, int32_t F, const moe_dropout_spec* spec, const void* a,
                         int64_t lda, const void* b, int64_t ldb, void* h, hipStream_t stream);

/* Its gradient: with d = keep ? c dh : 0 and s = 1 / (1 + exp(-a)),
 *   da = d b s (1 + a (1 - s)) (b = 1 when NULL), db = d a s; 0 where dropped.
 *   dh [rows, F] dense; da, db [rows, F] out with row strides ldda / lddb; db NULL exactly
 *   when b is. */
moe_status moe_gated_act_grad(int32_t dtype, int64_t rows, int32_t F, const moe_dropout_spec* spec,
                              const void* dh, const void* a, int64_t lda, const void* b, int64_t ldb, void* da,
                              int64_t ldda, void* db, int64_t lddb, hipStream_t stream);

/* The gradient of moe_combine:  dy_perm[row_of_pair[p]] = topk_w[p] * dout[p div k],
 * dtopk_w[p] = <dout[p div k], y_perm[row_of_pair[p]]>.  Pairs with a row below 0 or not
 * below `rows` were dropped: dtopk_w is 0 and no row is written.  Rows of dy_perm that no
 * pair names are left as they were.  No two pairs may name one row.
 *   dout [T, H], y_perm and dy_perm [rows, H] dtype; row_of_pair, topk_w, dtopk_w [T, k]
 *   (int32, fp32, fp32).  H a multiple of 8, 1 <= k <= 8, T < 2^24, rows < 2^31. */
moe_status moe_combine_grad(int32_t dtype, int64_t T, int32_t k, int32_t H, int64_t rows, const void* dout,
                            const void* y_perm, const int32_t* row_of_pair, const float* topk_w, void* dy_perm,
                            float* dtopk_w, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
