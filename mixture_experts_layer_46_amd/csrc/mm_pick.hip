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

const Cost* costs(int kind, int dtype) {
    if (kind == 3) return kInt8;
    if (dtype == MOE_F32) return kind == 2 ? kDw32 : kRows32;
    return kind == 0 ? kY16 : kind == 1 ? kDx16 : kDw16;
}

long long blocks_of(int kind, const MmArgs& a, const Shape& s) {
    const long long J = kind == 1 ? a.K : a.N;
    const long long ni = kind == 2 ? (long long)a.E * ((a.K + s.bm - 1) / s.bm)
                                   : ((long long)a.rows + s.bm - 1) / s.bm + std::min(a.rows, a.E);
    return ni * ((J + s.bn - 1) / s.bn);
}

// A launch holds at most 2^32 threads in a dimension.
bool fits(int kind, const MmArgs& a, int form) { return blocks_of(kind, a, kShape[form]) * kShape[form].threads < (1ll << 32); }

double estimate(int kind, int dtype, const MmArgs& a, int form, int cus) {
    const Shape& s = kShape[form];
    const Cost& c = costs(kind, dtype)[form];
    const int es = kind == 3 ? 1 : dtype == MOE_F32 ? 4 : 2;
    const double E = a.E, K = a.K, N = a.N, R = std::max(a.rows, 1);
    const double groups = std::min(E, R), mean = R / groups;             // groups that can have rows
    const double J = kind == 1 ? K : N, C = kind == 1 ? N : kind == 2 ? mean : K;
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
    const double bytes = (R * K + R * N) * es + (kind == 2 ? E : groups) * K * N * es, m = bytes / (kind == 2 ? kWriteRate : s.rate);
    return std::max(t, m) + .2 * std::min(t, m);
}

}  // namespace

bool mm_fits(int kind, int dtype, const MmArgs& a) {
    for (int f = 0; f < FORMS; ++f)
        if (costs(kind, dtype)[f].fixed != 0 && fits(kind, a, f)) return true;
    return false;
}

namespace {

// the form with the shortest estimate, or -1: mm_fits refuses such calls before
int pick(int kind, int dtype, const MmArgs& a, int cus) {
    int best = -1;
    double t_best = 0;
    for (int f = 0; f < FORMS; ++f) {
        if (costs(kind, dtype)[f].fixed == 0 || !fits(kind, a, f)) continue;
        const double t = estimate(kind, dtype, a, f, cus);
        if (best < 0 || t < t_best) best = f, t_best = t;
    }
    return best;
}

}  // namespace

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
