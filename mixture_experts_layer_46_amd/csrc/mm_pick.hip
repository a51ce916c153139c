// Which form of the grouped products' kernels a call takes (mm.hip and mm_stream.hip, mm_mid.hip,
// mm_thin.hip).
//
// The group sizes stay on the device, so the choice is made from what the host knows: the
// rows, the groups and the matrix sizes.  Each form's time is estimated as rounds of
// workgroups over the card's CUs, a round costing a fixed part plus its steps of 64 bytes,
// each step the larger of its latency when a workgroup is alone and of its share of a full
// CU; the bytes that every form has to move bound the whole from below.
//
// The three constants of a form come from some 12000 random calls (1-256 groups, 1-60000 rows,
// matrices of 64-8192 by 64-16384, even, Zipf and gapped loads), each timed in every form.
// Over 11000 further calls the form picked is slower than the best one by 1.4% (x W), 2.0% (dy
// W^T), 2.9% (x^T dy), 1.7% (int8) and 1.0% (fp32) in the geometric mean; the best single form
// would be 23%, 20%, 16%, 15% and 24% slower.  fp32 has no tiles of 128: they won
// 0.05% (weight gradients 0.6%) over the other forms.  The thin form of a weight gradient
// wins where one or two groups have small matrices: over such calls 6% (16 bits) and 18%
// (fp32) in the mean, at most 2.3 times.
#include <algorithm>
#include <cmath>

#include "common.h"
#include "launch.h"
#include "mm_launch.h"

namespace moe {

namespace {

enum Form { LARGE, MID128, MID64, THIN32, THIN16, FORMS };

struct Shape {
    int bm, bn;           // tile
    int per_cu;           // workgroups that a CU is taken to hold at once (see below)
    int split;            // wavefronts that share the contraction
    int threads;
    double rate;          // bytes per us that it reaches when weights streamed once are all there is
};
// per_cu is the model's, and the constants were fitted with it: what a CU's 160 KB of LDS hold
// is 1, 2, 3 (fp32: 4), 2 and 1 of these workgroups (135, 67, 51 (35), 75 and 123 KB each).
constexpr Shape kShape[FORMS] = {{256, 256, 1, 1, 512, 5.0e6}, {128, 128, 2, 1, 256, 5.3e6}, {64, 64, 4, 1, 256, 5.4e6},
                                 {32, 64, 2, 4, 256, 5.6e6},   {16, 64, 1, 8, 512, 4.9e6}};

struct Cost {
    double fixed, step, busy;     // us: per workgroup; per step alone; per step and workgroup of a full CU
};
// the forms that do not exist (fp32 LARGE and MID128, weight gradients in THIN16) have no cost
constexpr Cost kY16[FORMS] = {{1.85, .38, .54}, {1.9, .38, .25}, {2.15, .24, .146}, {2.15, .23, .59}, {3.55, .89, .042}};
constexpr Cost kDx16[FORMS] = {{1.85, .38, .59}, {1.8, .385, .24}, {1.85, .096, .14}, {3.75, .25, .34}, {2.55, .69, .039}};
constexpr Cost kDw16[FORMS] = {{3.4, .52, 1.0}, {2.1, .34, .28}, {2.0, .20, .116}, {1.5, .20, .55}, {}};
constexpr Cost kInt8[FORMS] = {{3.0, .33, .68}, {2.0, .44, .24}, {2.2, .21, .118}, {2.25, .25, .48}, {2.5, .69, .05}};
constexpr Cost kRows32[FORMS] = {{}, {}, {1.05, .52, .10}, {3.95, .545, .45}, {2.15, .96, .187}};
constexpr Cost kDw32[FORMS] = {{}, {}, {1.5, .68, .30}, {2.95, .44, .57}, {}};
constexpr double kWriteRate = 5.2e6;      // bytes per us of a weight gradient, in every form

// The kinds of mm_launch.h have shapes and costs of their own, fitted in the same way to random
// calls of 1-256 groups, 1-60000 rows, 64-8192 by 64-16384, timed in every form with the operands
// of successive calls at different places, so that weights come from memory.  Over 8100 to 9300
// calls each (fp8 18800, with fp32 output 92000), a part of them those of the fit, the form picked is
// slower than the best one by 1.4% (gated), 1.3% (gated, fp32), 3.2% (two-pair dx), 2.0% (fp32),
// 1.9% (fp8) and 0.9% (fp8, fp32 output); the best single form would be 11%, 27%, 22%, 17%, 19%
// and 18% slower.  A pair of weight gradients in one launch is estimated as one of them; and the
// forms are not compared with two products and the activation.  fp8 has no 16-row form with bf16 output:
// it was the best one in 4% of the calls and its choice won nothing.  (A gated tile's columns are
// those of h.)
struct FormCost {
    Shape s;
    Cost c;
};
constexpr FormCost kGated16[FORMS] = {
    {{256, 128, 1, 1, 512, 5.0e6}, {15.3, .395, .30}}, {{128, 64, 2, 1, 256, 6.5e6}, {3.93, .362, .281}},
    {{64, 64, 4, 1, 256, 6.5e6}, {3.54, .293, .196}},  {{32, 64, 2, 4, 256, 5.5e6}, {5.38, .30, .706}},
    {{16, 64, 1, 4, 256, 4.5e6}, {4.20, .321, .456}}};
constexpr FormCost kGated32[FORMS] = {
    {}, {}, {{64, 64, 2, 1, 256, 6.5e6}, {4.10, .426, .23}}, {{32, 64, 2, 4, 256, 6.5e6}, {4.69, .775, .894}},
    {{16, 64, 1, 4, 256, 5.0e6}, {5.07, .486, .30}}};
constexpr FormCost kTwo16[FORMS] = {
    {{256, 256, 1, 1, 512, 4.5e6}, {8.80, .559, .30}}, {{128, 128, 2, 1, 256, 5.0e6}, {3.61, .273, .274}},
    {{64, 64, 4, 1, 256, 5.5e6}, {3.31, .122, .112}},  {{32, 64, 2, 4, 256, 5.5e6}, {3.21, .293, .339}},
    {{16, 64, 1, 8, 512, 4.5e6}, {4.11, .369, .30}}};
constexpr FormCost kTwo32[FORMS] = {
    {}, {}, {{64, 64, 2, 1, 256, 6.5e6}, {3.38, .233, .133}}, {{32, 64, 2, 4, 256, 6.0e6}, {3.86, .326, .51}},
    {{16, 64, 1, 8, 512, 4.5e6}, {4.13, .559, .30}}};
constexpr FormCost kFp8[FORMS] = {
    {{256, 256, 1, 1, 512, 4.5e6}, {9.95, .486, .30}}, {{128, 128, 2, 1, 256, 5.0e6}, {3.81, .266, .257}},
    {{64, 64, 3, 1, 256, 5.0e6}, {3.71, .15, .128}},   {{32, 64, 2, 4, 256, 5.0e6}, {4.57, .291, .376}}, {}};
constexpr FormCost kFp8F32[FORMS] = {
    {}, {{128, 128, 2, 1, 256, 6.5e6}, {3.36, .60, .269}}, {{64, 64, 4, 1, 256, 5.5e6}, {3.67, .212, .19}},
    {{32, 64, 2, 4, 256, 6.5e6}, {5.27, .337, .392}}, {{16, 64, 1, 8, 512, 4.5e6}, {5.02, .452, .30}}};

FormCost form_of(int kind, int dtype, int form) {
    const bool f = dtype == MOE_F32;
    switch (kind) {
        case MM_FP8: return kFp8[form];
        case MM_FP8_F32: return kFp8F32[form];
        case MM_GATED: return f ? kGated32[form] : kGated16[form];
        case MM_DX_TWO: return f ? kTwo32[form] : kTwo16[form];
        case 3: return {kShape[form], kInt8[form]};
    }
    if (f) return {kShape[form], kind == 2 ? kDw32[form] : kRows32[form]};
    return {kShape[form], kind == 0 ? kY16[form] : kind == 1 ? kDx16[form] : kDw16[form]};
}

long long blocks_of(int kind, const MmArgs& a, const Shape& s) {
    const long long J = kind == 1 || kind == MM_DX_TWO ? a.K : a.N;
    const long long ni = kind == 2 ? (long long)a.E * ((a.K + s.bm - 1) / s.bm)
                                   : ((long long)a.rows + s.bm - 1) / s.bm + std::min(a.rows, a.E);
    return ni * ((J + s.bn - 1) / s.bn);
}

// Whether the form exists, and a launch (at most 2^32 threads) can hold the call's workgroups.
bool fits(int kind, const FormCost& f, const MmArgs& a) {
    return f.c.fixed != 0 && blocks_of(kind, a, f.s) * f.s.threads < (1ll << 32);
}

double estimate(int kind, int dtype, const MmArgs& a, const FormCost& f, int cus) {
    const Shape& s = f.s;
    const Cost& c = f.c;
    const bool dx = kind == 1 || kind == MM_DX_TWO;
    const int es = kind == 3 || kind == MM_FP8 || kind == MM_FP8_F32 ? 1 : dtype == MOE_F32 ? 4 : 2;
    const double E = a.E, K = a.K, N = a.N, R = std::max(a.rows, 1);
    const double groups = std::min(E, R), mean = R / groups;             // groups that can have rows
    const double J = dx ? K : N, C = kind == MM_DX_TWO ? 2 * N : dx ? N : kind == 2 ? mean : K;
    double tiles;                                                        // expected row tiles
    if (kind == 2) tiles = E * std::ceil(K / s.bm);
    else if (a.E == 1) tiles = std::ceil(R / s.bm);
    else tiles = mean > .75 * s.bm ? groups * std::max(1., mean / s.bm + .5) : groups;
    const double per_cu = tiles * std::ceil(J / s.bn) / cus;
    const double steps = std::ceil(std::ceil(C * es / 64) / s.split);
    double t;
    if (per_cu <= s.per_cu) {
        t = c.fixed + steps * std::max(c.step, std::ceil(per_cu) * c.busy);
    } else {
        const double r = per_cu / s.per_cu;
        t = (r < 2 ? 2 : r + .4) * (c.fixed + steps * std::max(c.step, s.per_cu * c.busy));
    }
    const double mats = kind == 2 ? E : kind == MM_GATED || kind == MM_DX_TWO ? 2 * groups : groups;
    const double bytes = (R * K + R * N * (kind == MM_DX_TWO ? 2 : 1)) * es + mats * K * N * es, m = bytes / (kind == 2 ? kWriteRate : s.rate);
    return std::max(t, m) + .2 * std::min(t, m);
}

}  // namespace

bool mm_fp8_fits(int out_dtype, const MmArgs& a) { return mm_fits(out_dtype == MOE_F32 ? MM_FP8_F32 : MM_FP8, MOE_BF16, a); }

bool mm_fits(int kind, int dtype, const MmArgs& a) {
    for (int f = 0; f < FORMS; ++f)
        if (fits(kind, form_of(kind, dtype, f), a)) return true;
    return false;
}

namespace {

// the form with the shortest estimate, or -1: mm_fits refuses such calls before
int pick(int kind, int dtype, const MmArgs& a, int cus) {
    int best = -1;
    double t_best = 0;
    for (int f = 0; f < FORMS; ++f) {
        const FormCost form = form_of(kind, dtype, f);
        if (!fits(kind, form, a)) continue;
        const double t = estimate(kind, dtype, a, form, cus);
        if (best < 0 || t < t_best) best = f, t_best = t;
    }
    return best;
}

}  // namespace

const char* mm_fp8_form(int out_dtype, const MmArgs& a, int cus) {
    return mm_form(out_dtype == MOE_F32 ? MM_FP8_F32 : MM_FP8, MOE_BF16, a, cus);
}

const char* mm_form(int kind, int dtype, const MmArgs& a, int cus) {
    switch (pick(kind, dtype, a, cus)) {
        case LARGE: return kind == 2 && mm_streams(a) ? "256x256 stream" : "256x256";
        case MID128: return "128x128";
        case MID64: return "64x64";
        case THIN32: return "32x64 thin";
        case THIN16: return "16x64 thin";
    }
    return nullptr;
}

hipError_t launch_mm_fp8(int out_dtype, const Fp8Args& a, hipStream_t st) {
    const int kind = out_dtype == MOE_F32 ? MM_FP8_F32 : MM_FP8;
    switch (pick(kind, MOE_BF16, a.m, device_cu_count())) {
        case LARGE: return launch_fp8_large(a, st);
        case MID128: return kind == MM_FP8 ? launch_fp8_mid(128, a, st) : launch_fp8_exact(128, a, st);
        case MID64: return kind == MM_FP8 ? launch_fp8_mid(64, a, st) : launch_fp8_exact(64, a, st);
        case THIN32: return launch_fp8_thin(32, out_dtype, a, st);
        case THIN16: return launch_fp8_thin(16, out_dtype, a, st);     // fp32 output
    }
    return hipErrorInvalidConfiguration;
}

hipError_t launch_mm(int kind, int dtype, int out_dtype, const MmArgs& a, hipStream_t st) {
    switch (pick(kind, dtype, a, device_cu_count())) {
        case LARGE: return launch_mm_large(kind, out_dtype, a, st);
        case MID128: return launch_mm_mid(128, kind, dtype, out_dtype, a, st);
        case MID64: return launch_mm_mid(64, kind, dtype, out_dtype, a, st);
        case THIN32: return launch_mm_thin(32, kind, dtype, out_dtype, a, st);
        case THIN16: return launch_mm_thin(16, kind, dtype, out_dtype, a, st);
    }
    return hipErrorInvalidConfiguration;
}

}  // namespace moe
