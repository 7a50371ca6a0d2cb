// Helpers of the policy loss's kernels
#pragma once
#include "iqlher.h"
#include "launch.hpp"
#include "tile16.hpp"

namespace iqlh {
namespace policy {

constexpr int kNT = 256;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kNone = -__builtin_huge_valf();

// 2^(x - m); 0 for x of minus infinity, whatever m is
IQLH_DEV float exp_below(float x, float m) { return x == kNone ? 0.f : __builtin_amdgcn_exp2f(x - m); }

// Maximum of logits times log2(e), and sum of 2^(. - maximum)
struct Soft {
    float m, s;
    IQLH_DEV void join(Soft o) {
        const float top = fmaxf(m, o.m);
        s = s * exp_below(m, top) + o.s * exp_below(o.m, top);  // NaN stays NaN
        m = top;
    }
};
IQLH_DEV Soft soft_xor(Soft v, int lanes) {
    v.join(Soft{__shfl_xor(v.m, lanes, kWave), __shfl_xor(v.s, lanes, kWave)});
    return v;
}

// A row that adds nothing: no action, or none of these, or weight 0
IQLH_DEV bool row_off(const int32_t* taken, const float* row_weights, int64_t actions, int64_t m) {
    const int32_t t = taken[m];
    return t < 0 || t >= actions || (row_weights && row_weights[m] == 0.f);
}

struct FinishArgs {
    const Soft* part;        // [parts][rows]
    const float* z_taken;
    const int32_t* taken;
    const float* row_weights;
    float* nll;
    float* lse;
    float* loss;             // or null
    double* loss_part;       // [workgroups]
    int32_t* flags;
    int64_t rows, actions;
    int parts;
    double scale;
};
IQLH_DEV void put_loss(const FinishArgs& a, double sum) {
    const float loss = (float)(sum * a.scale);
    if (a.loss) *a.loss = loss;
    if (!(fabsf(loss) < __uint_as_float(0x7F800000u))) set_flag(a.flags, IQLH_FLAG_NONFINITE_LOSS);
}
}  // namespace policy
}  // namespace iqlh
