// What the kernels of orthogonalised updates share
#pragma once
#include <math.h>

#include "common.hpp"

namespace iqlh {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kUp = 8192.f, kDown = 1.f / 8192.f;  // of every operand

// X is held times 2^e, e >= 0, so that a norm far below eps leaves it its bits.  e of an update of this norm, X's
// being norm / (norm + eps), which 2^e takes to [1/2, 1)
IQLH_DEV int32_t ortho_exponent(double norm, double eps) {
    int e = 0;
    (void)frexp(norm / (norm + eps), &e);
    return e >= 0 ? 0 : e < -120 ? 120 : -e;  // norms down to 2^-120 of eps
}
// e after `step` steps: a step takes X's norm up by a = 3.4445 < 2^(29/16) at most, so 2^e |X| stays below 1 or e is 0
IQLH_DEV int32_t ortho_exponent_at(int32_t e, int32_t step) {
    const int32_t left = e - (29 * step + 15) / 16;
    return left > 0 ? left : 0;
}
// (1 - decay) w - rate x in two multiply-adds; an infinite w stays one
IQLH_DEV float ortho_weight(float w, float x, float rate, float decay) {
    const float y = fmaf(-decay, w, fmaf(-rate, x, w));
    return fabsf(w) == __builtin_huge_valf() ? (1.f - decay) * w : y;
}
// s of the weights' update
IQLH_DEV double ortho_shape(int rows, int cols, int scale) {
    const double r = rows, c = cols;
    return scale == 0 ? sqrt(r > c ? r / c : 1.0) : 0.2 * sqrt(r > c ? r : c);  // IQLH_MUON_SCALE_SHAPE, _RMS
}

}  // namespace iqlh
