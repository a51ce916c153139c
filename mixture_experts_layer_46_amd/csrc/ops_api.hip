// C ABI of the training and 8-bit operators: argument checks and launches.
// Declarations, argument meaning, layouts and limits: include/moe_ops.h.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "common.h"
#include "launch.h"
#include "mm_launch.h"
#include "moe_ops.h"

namespace moe {

namespace {

moe_status fail(moe_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return report_error(st, buf);
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

#define REQ(p, name)                                                     \
    do {                                                                 \
        if (!(p)) return fail(MOE_ERR_NULL, "%s is NULL", name);         \
        if (!aligned16(p)) return fail(MOE_ERR_ALIGN, "%s is not 16-byte aligned", name); \
    } while (0)
#define CHECK(expr)                                                      \
    do {                                                                 \
        const moe_status st_ = (expr);                                   \
        if (st_ != MOE_OK) return st_;                                   \
    } while (0)
#define HIPCHK(expr, where)                                              \
    do {                                                                 \
        (void)hipGetLastError();                                         \
        const hipError_t e_ = (expr);                                    \
        if (e_ != hipSuccess) return fail(MOE_ERR_HIP, "%s: %s", where, hipGetErrorString(e_)); \
    } while (0)

constexpr int kMaxDim = 1 << 20;          // K, N: 256 rows of fp32 stay below 2 GiB
constexpr int kMaxInt8K = 131056;         // 128 * 128 * K < 2^31
constexpr int64_t kMaxGrid = 1 << 24;     // workgroups of 256 threads: 2^32 work items a launch
constexpr int64_t kMaxElems = 1ll << 34;
constexpr int kMaxNorm = 16384;           // a row stays in a workgroup's registers

moe_status check_dtype(int32_t dtype) {
    if (dtype != MOE_F32 && dtype != MOE_BF16) return fail(MOE_ERR_UNSUPPORTED, "dtype %d unknown", dtype);
    return MOE_OK;
}

// `int8`: the 8-bit product (own limits, dtype ignored); `dw`: the weight gradient (fp32
// output of bf16 operands allowed)
moe_status check_mm(const moe_mm_shape* s, bool int8, bool dw) {
    if (!s) return fail(MOE_ERR_NULL, "shape is NULL");
    if (s->rows < 0) return fail(MOE_ERR_SHAPE, "rows = %lld < 0", (long long)s->rows);
    if (s->E <= 0 || s->K <= 0 || s->N <= 0)
        return fail(MOE_ERR_SHAPE, "E, K, N must be positive (E=%d K=%d N=%d)", s->E, s->K, s->N);
    if (s->E > 256) return fail(MOE_ERR_UNSUPPORTED, "E = %d > 256 is not supported", s->E);
    if (s->K % 8 || s->N % 8)
        return fail(MOE_ERR_UNSUPPORTED, "K and N must be multiples of 8 (K=%d N=%d)", s->K, s->N);
    if (s->K > kMaxDim || s->N > kMaxDim) return fail(MOE_ERR_UNSUPPORTED, "K=%d or N=%d above 2^20", s->K, s->N);
    if (s->rows >= 64 * kMaxGrid) return fail(MOE_ERR_UNSUPPORTED, "rows = %lld >= 2^30", (long long)s->rows);
    if (s->flags & ~MOE_MM_ZERO_REST) return fail(MOE_ERR_UNSUPPORTED, "unknown flag bits 0x%x", s->flags);
    if (int8) {
        if (s->K % 16) return fail(MOE_ERR_UNSUPPORTED, "int8: K must be a multiple of 16 (K=%d)", s->K);
        if (s->K > kMaxInt8K) return fail(MOE_ERR_UNSUPPORTED, "int8: K=%d above %d", s->K, kMaxInt8K);
        return check_dtype(s->out_dtype);
    }
    CHECK(check_dtype(s->dtype));
    CHECK(check_dtype(s->out_dtype));
    if (s->out_dtype != s->dtype && !(dw && s->dtype == MOE_BF16))
        return fail(MOE_ERR_UNSUPPORTED, "output type %d for operands of type %d", s->out_dtype, s->dtype);
    return MOE_OK;
}

moe_status check_fp8(const moe_mm_shape* s) {
    moe_mm_shape t = s ? *s : moe_mm_shape{};
    t.dtype = t.out_dtype;                    // the operands' type is no choice
    CHECK(check_mm(s ? &t : nullptr, false, false));
    if (s->K % 16) return fail(MOE_ERR_UNSUPPORTED, "fp8: K must be a multiple of 16 (K=%d)", s->K);
    return MOE_OK;
}

MmArgs mm_args(const moe_mm_shape& s, const void* a, const void* b, void* c, const int32_t* offsets) {
    return MmArgs{a, b, c, offsets, nullptr, nullptr, (int)s.rows, s.E, s.K, s.N, (s.flags & MOE_MM_ZERO_REST) ? 1 : 0};
}

moe_status check_spec(const moe_dropout_spec* spec, DropArgs* d) {
    if (!spec) return fail(MOE_ERR_NULL, "spec is NULL");
    if (!(spec->p >= 0.0 && spec->p <= 1.0)) return fail(MOE_ERR_SHAPE, "p = %g must lie in [0, 1]", spec->p);
    if ((uintptr_t)spec->step_device & 7u) return fail(MOE_ERR_ALIGN, "step_device is not 8-byte aligned");
    const uint32_t thr = (uint32_t)std::nearbyint(spec->p * 65536.0);
    *d = DropArgs{thr, thr < 65536 ? (float)(65536.0 / (65536.0 - thr)) : 0.f, spec->seed, spec->step, spec->step_device};
    return MOE_OK;
}

moe_status check_act(int32_t dtype, int64_t rows, int32_t F) {
    CHECK(check_dtype(dtype));
    if (rows < 0) return fail(MOE_ERR_SHAPE, "rows = %lld < 0", (long long)rows);
    if (F <= 0) return fail(MOE_ERR_SHAPE, "F = %d must be positive", F);
    if (F % 8) return fail(MOE_ERR_UNSUPPORTED, "F = %d must be a multiple of 8", F);
    if (rows >= kMaxElems / F) return fail(MOE_ERR_UNSUPPORTED, "rows * F = %lld * %d >= 2^34", (long long)rows, F);
    return MOE_OK;
}
moe_status check_ld(int64_t ld, int32_t F, const char* name) {
    if (ld < F) return fail(MOE_ERR_SHAPE, "%s = %lld < F = %d", name, (long long)ld, F);
    if (ld % 8) return fail(MOE_ERR_UNSUPPORTED, "%s = %lld must be a multiple of 8", name, (long long)ld);
    if (ld >= (1ll << 31)) return fail(MOE_ERR_UNSUPPORTED, "%s = %lld >= 2^31", name, (long long)ld);
    return MOE_OK;
}

moe_status too_many(const moe_mm_shape& s, const char* where) {
    return fail(MOE_ERR_UNSUPPORTED, "%s: too many output tiles for one launch (rows=%lld E=%d K=%d N=%d)", where,
                (long long)s.rows, s.E, s.K, s.N);
}

// `kind` is a moe_mm_product, and one of the kinds of mm_tile.h, or one of mm_launch.h's
moe_status run_mm(int kind, const moe_mm_shape& s, const MmArgs& a, hipStream_t st, const char* where) {
    if (!mm_fits(kind, s.dtype, a)) return too_many(s, where);
    HIPCHK(launch_mm(kind, s.dtype, s.out_dtype, a, st), where);
    return MOE_OK;
}

moe_status check_norm(const moe_norm_shape* s, const void* z, const float* w_post, const float* gate,
                      const float* w_next) {
    if (!s) return fail(MOE_ERR_NULL, "shape is NULL");
    CHECK(check_dtype(s->dtype));
    if (s->T < 0) return fail(MOE_ERR_SHAPE, "T = %lld < 0", (long long)s->T);
    if (s->T >= (1ll << 31)) return fail(MOE_ERR_UNSUPPORTED, "T = %lld >= 2^31", (long long)s->T);
    if (s->H <= 0) return fail(MOE_ERR_SHAPE, "H = %d must be positive", s->H);
    if (s->H % 8 || s->H > kMaxNorm)
        return fail(MOE_ERR_UNSUPPORTED, "H = %d must be a multiple of 8, at most %d", s->H, kMaxNorm);
    if (!(s->eps > 0.f && s->eps < INFINITY)) return fail(MOE_ERR_SHAPE, "eps = %g must be positive", (double)s->eps);
    if (!std::isfinite(s->scale)) return fail(MOE_ERR_SHAPE, "scale = %g must be finite", (double)s->scale);
    CHECK(check_ld(s->ldx, s->H, "ldx"));
    if (s->gate < MOE_GATE_NONE || s->gate > MOE_GATE_TOKEN)
        return fail(MOE_ERR_UNSUPPORTED, "gate kind %d unknown", s->gate);
    if (s->T > 0 && (gate != nullptr) != (s->gate != MOE_GATE_NONE))
        return fail(MOE_ERR_NULL, "gate and its kind (%d) do not match", s->gate);
    if (z) {
        CHECK(check_ld(s->ldz, s->H, "ldz"));
    } else if (s->T > 0) {
        if (w_post || gate) return fail(MOE_ERR_NULL, "w_post and gate need z");
        if (!w_next) return fail(MOE_ERR_NULL, "w_next is NULL");
    }
    return MOE_OK;
}
NormArgs norm_args(const moe_norm_shape& s, const void* x, const void* z, const float* w_post, const float* gate,
                   const float* w_next, void* y, void* u) {
    return NormArgs{x, z, w_post, gate, w_next, y, u, (long long)s.T, (long long)s.ldx, (long long)s.ldz, s.H, s.gate, s.scale, s.eps};
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_grouped_mm(const moe_mm_shape* shape, const void* x, const void* w, const int32_t* offsets, void* y,
                          hipStream_t stream) {
    CHECK(check_mm(shape, false, false));
    if (shape->rows == 0) return MOE_OK;
    REQ(x, "x");
    REQ(w, "w");
    REQ(offsets, "offsets");
    REQ(y, "y");
    return run_mm(MOE_MM_Y, *shape, mm_args(*shape, x, w, y, offsets), stream, "grouped_mm");
}

moe_status moe_grouped_mm_dx(const moe_mm_shape* shape, const void* dy, const void* w, const int32_t* offsets, void* dx,
                             hipStream_t stream) {
    CHECK(check_mm(shape, false, false));
    if (shape->rows == 0) return MOE_OK;
    REQ(dy, "dy");
    REQ(w, "w");
    REQ(offsets, "offsets");
    REQ(dx, "dx");
    return run_mm(MOE_MM_DX, *shape, mm_args(*shape, dy, w, dx, offsets), stream, "grouped_mm_dx");
}

moe_status moe_grouped_mm_dw(const moe_mm_shape* shape, const void* x, const void* dy, const int32_t* offsets, void* dw,
                             hipStream_t stream) {
    CHECK(check_mm(shape, false, true));
    if (shape->rows > 0) {
        REQ(x, "x");
        REQ(dy, "dy");
    }
    REQ(offsets, "offsets");
    REQ(dw, "dw");
    return run_mm(MOE_MM_DW, *shape, mm_args(*shape, x, dy, dw, offsets), stream, "grouped_mm_dw");
}

const char* moe_grouped_mm_form(const moe_mm_shape* shape, int32_t product, int32_t cus) {
    if (product < MOE_MM_Y || product > MOE_MM_INT8) return fail(MOE_ERR_SHAPE, "product %d unknown", product), nullptr;
    if (cus < 0) return fail(MOE_ERR_SHAPE, "cus = %d < 0", cus), nullptr;
    if (check_mm(shape, product == MOE_MM_INT8, product == MOE_MM_DW) != MOE_OK) return nullptr;
    const MmArgs a = mm_args(*shape, nullptr, nullptr, nullptr, nullptr);
    if (!mm_fits(product, shape->dtype, a)) return too_many(*shape, "grouped_mm_form"), nullptr;
    return mm_form(product, shape->dtype, a, cus ? cus : device_cu_count());
}

moe_status moe_gated_mm(const moe_mm_shape* shape, const void* x, const void* w_in, const void* w_up, const int32_t* offsets,
                        void* h, void* a, void* b, hipStream_t stream) {
    CHECK(check_mm(shape, false, false));
    if (shape->rows == 0) return MOE_OK;
    REQ(x, "x");
    REQ(w_in, "w_in");
    REQ(w_up, "w_up");
    REQ(offsets, "offsets");
    REQ(h, "h");
    if ((a != nullptr) != (b != nullptr)) return fail(MOE_ERR_NULL, "a and b must be given together");
    if (a) {
        REQ(a, "a");
        REQ(b, "b");
    }
    MmArgs m = mm_args(*shape, x, w_in, h, offsets);
    m.b2 = w_up;
    m.ca = a;
    m.cb = b;
    return run_mm(MM_GATED, *shape, m, stream, "gated_mm");
}

moe_status moe_gated_mm_dx(const moe_mm_shape* shape, const void* da, const void* db, const void* w_in, const void* w_up,
                           const int32_t* offsets, void* dx, hipStream_t stream) {
    CHECK(check_mm(shape, false, false));
    if (shape->rows == 0) return MOE_OK;
    REQ(da, "da");
    REQ(db, "db");
    REQ(w_in, "w_in");
    REQ(w_up, "w_up");
    REQ(offsets, "offsets");
    REQ(dx, "dx");
    MmArgs m = mm_args(*shape, da, w_in, dx, offsets);
    m.a2 = db;
    m.b2 = w_up;
    return run_mm(MM_DX_TWO, *shape, m, stream, "gated_mm_dx");
}

moe_status moe_gated_mm_dw(const moe_mm_shape* shape, const void* x, const void* da, const void* db, const int32_t* offsets,
                           void* dw_in, void* dw_up, hipStream_t stream) {
    CHECK(check_mm(shape, false, true));
    if (shape->rows > 0) {
        REQ(x, "x");
        REQ(da, "da");
        REQ(db, "db");
    }
    REQ(offsets, "offsets");
    REQ(dw_in, "dw_in");
    REQ(dw_up, "dw_up");
    MmArgs m = mm_args(*shape, x, da, dw_in, offsets);
    m.b2 = shape->rows > 0 ? db : offsets;    // not NULL, and not read without rows
    m.ca = dw_up;
    return run_mm(MOE_MM_DW, *shape, m, stream, "gated_mm_dw");
}

const char* moe_gated_mm_form(const moe_mm_shape* shape, int32_t dx, int32_t cus) {
    if (cus < 0) return fail(MOE_ERR_SHAPE, "cus = %d < 0", cus), nullptr;
    if (check_mm(shape, false, false) != MOE_OK) return nullptr;
    const MmArgs a = mm_args(*shape, nullptr, nullptr, nullptr, nullptr);
    const int kind = dx ? MM_DX_TWO : MM_GATED;
    if (!mm_fits(kind, shape->dtype, a)) return too_many(*shape, "gated_mm_form"), nullptr;
    return mm_form(kind, shape->dtype, a, cus ? cus : device_cu_count());
}

moe_status moe_quantize_rows(int32_t dtype, int64_t rows, int32_t K, const void* x, int8_t* q, float* scale,
                             hipStream_t stream) {
    CHECK(check_dtype(dtype));
    if (rows < 0) return fail(MOE_ERR_SHAPE, "rows = %lld < 0", (long long)rows);
    if (K <= 0) return fail(MOE_ERR_SHAPE, "K = %d must be positive", K);
    if (K % 8 || K > kMaxDim) return fail(MOE_ERR_UNSUPPORTED, "K = %d must be a multiple of 8, at most 2^20", K);
    if (rows >= kMaxGrid) return fail(MOE_ERR_UNSUPPORTED, "rows = %lld >= 2^24", (long long)rows);
    if (rows == 0) return MOE_OK;
    REQ(x, "x");
    REQ(q, "q");
    REQ(scale, "scale");
    HIPCHK(launch_quantize_rows(x, dtype, rows, K, q, scale, stream), "quantize_rows");
    return MOE_OK;
}

moe_status moe_quantize_experts(int32_t dtype, int32_t E, int32_t K, int32_t N, const void* w, int8_t* q, float* scale,
                                hipStream_t stream) {
    CHECK(check_dtype(dtype));
    const moe_mm_shape s{0, E, K, N, dtype, dtype, 0};
    CHECK(check_mm(&s, true, false));
    REQ(w, "w");
    REQ(q, "q");
    REQ(scale, "scale");
    HIPCHK(launch_quantize_experts(w, dtype, E, K, N, q, scale, stream), "quantize_experts");
    return MOE_OK;
}

moe_status moe_grouped_mm_int8(const moe_mm_shape* shape, const int8_t* xq, const float* x_scale, const int8_t* wq,
                               const float* w_scale, const int32_t* offsets, void* y, hipStream_t stream) {
    CHECK(check_mm(shape, true, false));
    if (shape->rows == 0) return MOE_OK;
    REQ(xq, "xq");
    REQ(x_scale, "x_scale");
    REQ(wq, "wq");
    REQ(w_scale, "w_scale");
    REQ(offsets, "offsets");
    REQ(y, "y");
    MmArgs a = mm_args(*shape, xq, wq, y, offsets);
    a.xs = x_scale;
    a.ws = w_scale;
    return run_mm(MOE_MM_INT8, *shape, a, stream, "grouped_mm_int8");
}

moe_status moe_quantize_rows_fp8(int32_t dtype, int64_t rows, int32_t K, const void* x, uint8_t* q, uint8_t* scale,
                                 hipStream_t stream) {
    CHECK(check_dtype(dtype));
    if (rows < 0) return fail(MOE_ERR_SHAPE, "rows = %lld < 0", (long long)rows);
    if (K <= 0) return fail(MOE_ERR_SHAPE, "K = %d must be positive", K);
    if (K % 16 || K > kMaxDim) return fail(MOE_ERR_UNSUPPORTED, "K = %d must be a multiple of 16, at most 2^20", K);
    if (rows >= kMaxGrid) return fail(MOE_ERR_UNSUPPORTED, "rows = %lld >= 2^24", (long long)rows);
    if (rows == 0) return MOE_OK;
    REQ(x, "x");
    REQ(q, "q");
    REQ(scale, "scale");
    HIPCHK(launch_quantize_rows_fp8(x, dtype, rows, K, q, scale, stream), "quantize_rows_fp8");
    return MOE_OK;
}

moe_status moe_quantize_experts_fp8(int32_t dtype, int32_t E, int32_t K, int32_t N, const void* w, uint8_t* q,
                                    uint8_t* scale, hipStream_t stream) {
    CHECK(check_dtype(dtype));
    const moe_mm_shape s{0, E, K, N, dtype, dtype, 0};
    CHECK(check_fp8(&s));
    const long long blocks = (long long)E * ((K + 127) / 128) * ((N + 127) / 128);
    if (blocks >= kMaxGrid)
        return fail(MOE_ERR_UNSUPPORTED, "quantize_experts_fp8: %lld blocks, at most 2^24 (E=%d K=%d N=%d)", blocks, E, K, N);
    REQ(w, "w");
    REQ(q, "q");
    REQ(scale, "scale");
    HIPCHK(launch_quantize_experts_fp8(w, dtype, E, K, N, q, scale, stream), "quantize_experts_fp8");
    return MOE_OK;
}

moe_status moe_grouped_mm_fp8(const moe_mm_shape* shape, const uint8_t* xq, const uint8_t* x_scale, const uint8_t* wq,
                              const uint8_t* w_scale, const int32_t* offsets, void* y, hipStream_t stream) {
    CHECK(check_fp8(shape));
    if (shape->rows == 0) return MOE_OK;
    REQ(xq, "xq");
    REQ(x_scale, "x_scale");
    REQ(wq, "wq");
    REQ(w_scale, "w_scale");
    REQ(offsets, "offsets");
    REQ(y, "y");
    const Fp8Args a{mm_args(*shape, xq, wq, y, offsets), x_scale, w_scale};
    if (!mm_fp8_fits(shape->out_dtype, a.m)) return too_many(*shape, "grouped_mm_fp8");
    HIPCHK(launch_mm_fp8(shape->out_dtype, a, stream), "grouped_mm_fp8");
    return MOE_OK;
}

const char* moe_grouped_mm_fp8_form(const moe_mm_shape* shape, int32_t cus) {
    if (cus < 0) return fail(MOE_ERR_SHAPE, "cus = %d < 0", cus), nullptr;
    if (check_fp8(shape) != MOE_OK) return nullptr;
    const MmArgs a = mm_args(*shape, nullptr, nullptr, nullptr, nullptr);
    if (!mm_fp8_fits(shape->out_dtype, a)) return too_many(*shape, "grouped_mm_fp8_form"), nullptr;
    return mm_fp8_form(shape->out_dtype, a, cus ? cus : device_cu_count());
}

moe_status moe_dropout(int32_t dtype, int64_t n, const moe_dropout_spec* spec, const void* x, void* y,
                       hipStream_t stream) {
    CHECK(check_dtype(dtype));
    DropArgs d;
    CHECK(check_spec(spec, &d));
    if (n < 0) return fail(MOE_ERR_SHAPE, "n = %lld < 0", (long long)n);
    if (n >= kMaxElems) return fail(MOE_ERR_UNSUPPORTED, "n = %lld >= 2^34", (long long)n);
    if (n == 0) return MOE_OK;
    REQ(x, "x");
    REQ(y, "y");
    HIPCHK(launch_dropout(x, y, dtype, n, d, stream), "dropout");
    return MOE_OK;
}

moe_status moe_gated_act(int32_t dtype, int64_t rows, int32_t F, const moe_dropout_spec* spec, const void* a,
                         int64_t lda, const void* b, int64_t ldb, void* h, hipStream_t stream) {
    CHECK(check_act(dtype, rows, F));
    DropArgs d;
    CHECK(check_spec(spec, &d));
    CHECK(check_ld(lda, F, "lda"));
    if (b) CHECK(check_ld(ldb, F, "ldb"));
    if (rows == 0) return MOE_OK;
    REQ(a, "a");
    if (b) REQ(b, "b");
    REQ(h, "h");
    HIPCHK(launch_gated_act(a, lda, b, ldb, h, dtype, rows, F, d, stream), "gated_act");
    return MOE_OK;
}

moe_status moe_gated_act_grad(int32_t dtype, int64_t rows, int32_t F, const moe_dropout_spec* spec, const void* dh,
                              const void* a, int64_t lda, const void* b, int64_t ldb, void* da, int64_t ldda, void* db,
                              int64_t lddb, hipStream_t stream) {
    CHECK(check_act(dtype, rows, F));
    DropArgs d;
    CHECK(check_spec(spec, &d));
    CHECK(check_ld(lda, F, "lda"));
    CHECK(check_ld(ldda, F, "ldda"));
    if ((b == nullptr) != (db == nullptr) && rows > 0) return fail(MOE_ERR_NULL, "b and db must be given together");
    if (b) {
        CHECK(check_ld(ldb, F, "ldb"));
        CHECK(check_ld(lddb, F, "lddb"));
    }
    if (rows == 0) return MOE_OK;
    REQ(dh, "dh");
    REQ(a, "a");
    if (b) REQ(b, "b");
    REQ(da, "da");
    if (db) REQ(db, "db");
    HIPCHK(launch_gated_act_grad(dh, a, lda, b, ldb, da, ldda, db, lddb, dtype, rows, F, d, stream), "gated_act_grad");
    return MOE_OK;
}

moe_status moe_combine_grad(int32_t dtype, int64_t T, int32_t k, int32_t H, int64_t rows, const void* dout,
                            const void* y_perm, const int32_t* row_of_pair, const float* topk_w, void* dy_perm,
                            float* dtopk_w, hipStream_t stream) {
    CHECK(check_dtype(dtype));
    if (T < 0 || rows < 0) return fail(MOE_ERR_SHAPE, "T = %lld or rows = %lld < 0", (long long)T, (long long)rows);
    if (k <= 0 || H <= 0) return fail(MOE_ERR_SHAPE, "k, H must be positive (k=%d H=%d)", k, H);
    if (k > 8) return fail(MOE_ERR_UNSUPPORTED, "k = %d > 8 is not supported", k);
    if (H % 8) return fail(MOE_ERR_UNSUPPORTED, "H = %d must be a multiple of 8", H);
    if (T >= kMaxGrid) return fail(MOE_ERR_UNSUPPORTED, "T = %lld >= 2^24", (long long)T);
    if (rows >= (1ll << 31)) return fail(MOE_ERR_UNSUPPORTED, "rows = %lld >= 2^31", (long long)rows);
    if (T == 0) return MOE_OK;
    REQ(dout, "dout");
    if (rows > 0) {
        REQ(y_perm, "y_perm");
        REQ(dy_perm, "dy_perm");
    }
    REQ(row_of_pair, "row_of_pair");
    REQ(topk_w, "topk_w");
    REQ(dtopk_w, "dtopk_w");
    HIPCHK(launch_combine_grad(dout, y_perm, row_of_pair, topk_w, dy_perm, dtopk_w, T, k, H, dtype, rows, stream),
           "combine_grad");
    return MOE_OK;
}

moe_status moe_residual_norm(const moe_norm_shape* shape, const void* x, const void* z, const float* w_post,
                             const float* gate, const float* w_next, void* y, void* u, hipStream_t stream) {
    CHECK(check_norm(shape, z, w_post, gate, w_next));
    if (shape->T == 0) return MOE_OK;
    REQ(x, "x");
    if (z) {
        REQ(z, "z");
        REQ(y, "y");
    } else if (y) {
        return fail(MOE_ERR_NULL, "y needs z");
    }
    if ((u != nullptr) != (w_next != nullptr)) return fail(MOE_ERR_NULL, "w_next and u must be given together");
    if (w_post) REQ(w_post, "w_post");
    if (gate) REQ(gate, "gate");
    if (w_next) REQ(w_next, "w_next");
    if (u) REQ(u, "u");
    HIPCHK(launch_norm(norm_args(*shape, x, z, w_post, gate, w_next, y, u), shape->dtype, stream), "residual_norm");
    return MOE_OK;
}

moe_status moe_residual_norm_grad_workspace(const moe_norm_shape* shape, size_t* bytes) {
    if (!shape) return fail(MOE_ERR_NULL, "shape is NULL");
    if (!bytes) return fail(MOE_ERR_NULL, "bytes is NULL");
    if (shape->T < 0 || shape->T >= (1ll << 31) || shape->H <= 0 || shape->H % 8 || shape->H > kMaxNorm)
        return fail(MOE_ERR_SHAPE, "T = %lld or H = %d out of range", (long long)shape->T, shape->H);
    *bytes = (size_t)norm_grad_parts(shape->T, shape->H) * 3 * shape->H * sizeof(float);
    return MOE_OK;
}

moe_status moe_residual_norm_grad(const moe_norm_shape* shape, const void* dy, const void* du, const void* x,
                                  const void* z, const float* w_post, const float* gate, const float* w_next, void* dx,
                                  void* dz, float* dw_post, float* dgate, float* dw_next, void* workspace,
                                  size_t ws_bytes, hipStream_t stream) {
    CHECK(check_norm(shape, z, w_post, gate, w_next));
    if ((dw_post != nullptr) != (w_post != nullptr)) return fail(MOE_ERR_NULL, "w_post and dw_post must be given together");
    if ((dw_next != nullptr) != (w_next != nullptr)) return fail(MOE_ERR_NULL, "w_next and dw_next must be given together");
    if ((dgate != nullptr) != (gate != nullptr)) return fail(MOE_ERR_NULL, "gate and dgate must be given together");
    if (shape->T > 0) {
        REQ(x, "x");
        REQ(dx, "dx");
        if ((dz != nullptr) != (z != nullptr)) return fail(MOE_ERR_NULL, "z and dz must be given together");
        if (z) {
            REQ(z, "z");
            REQ(dz, "dz");
        } else if (dy) {
            return fail(MOE_ERR_NULL, "dy needs z");
        }
        if (dy) REQ(dy, "dy");
        if ((du != nullptr) != (w_next != nullptr)) return fail(MOE_ERR_NULL, "w_next and du must be given together");
        if (du) REQ(du, "du");
        if (w_post) REQ(w_post, "w_post");
        if (gate) REQ(gate, "gate");
        if (w_next) REQ(w_next, "w_next");
    }
    if (dw_post) REQ(dw_post, "dw_post");
    if (dgate) REQ(dgate, "dgate");
    if (dw_next) REQ(dw_next, "dw_next");
    const size_t need = (size_t)norm_grad_parts(shape->T, shape->H) * 3 * shape->H * sizeof(float);
    if (need) {
        REQ(workspace, "workspace");
        if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, need);
    }
    const NormGradArgs g{norm_args(*shape, x, z, w_post, gate, w_next, nullptr, nullptr), dy, du, dx, dz, dw_post, dgate,
                         dw_next, (float*)workspace};
    HIPCHK(launch_norm_grad(g, shape->dtype, stream), "residual_norm_grad");
    return MOE_OK;
}

}  // extern "C"
