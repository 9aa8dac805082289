// The softcap of scores to float32's accuracy, in base-2 units.
#pragma once

#include "ptx.cuh"

namespace flex {

constexpr float kLog2eF = 1.4426950408889634f;

// cap tanh(u), u = s / cap, in base-2 units.  From |u| = 1/4 on as cap (1 - 2 / (1
// + e^(2 u))), which is within 2^-22 cap: about 2^-20 of the result, but nothing
// of it where u is small.  There the Taylor series to u^9, which leaves out less
// than 2^-26 of it.  Together a tenth of tanhf's instructions.
// in = 2 log2(e) / cap, out = cap log2(e), both finite.
__device__ __forceinline__ float softcap_log2(float s, float in, float out) {
    constexpr double k = 0.69314718055994530942 * 0.69314718055994530942 / 4;  // u^2 = k z^2
    const float z = s * in, t = z * z;
    float near = fmaf(t, (float)(62. / 2835 * k * k * k * k), (float)(-17. / 315 * k * k * k));
    near = fmaf(t, near, (float)(2. / 15 * k * k));
    near = fmaf(t, near, (float)(-1. / 3 * k));
    near = fmaf(t, near, 1.f) * (s * kLog2eF);
    const float far = fmaf(out, -2.f * rcp_approx(1.f + ex2_approx(z)), out);
    return fabsf(z) < 0.5f * kLog2eF ? near : far;
}

}  // namespace flex
