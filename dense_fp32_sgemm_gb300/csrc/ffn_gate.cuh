// The gate's activation and its derivative, in FP32.
#pragma once

#include "ops_common.cuh"

namespace sgemm {

// ACCURATE: the exponential of the math library (FP32 results); else the
// hardware's, whose relative error of about 2^-21 at the sizes that matter is
// far below the 2^-9 or 2^-12 of a 16-bit result.
template <bool ACCURATE>
__device__ __forceinline__ float gate_exp(float x) {
    return ACCURATE ? expf(x) : __expf(x);
}
constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluK = 0.044715f;

// 1 / (1 + exp(-x)).  exp(-x) may reach infinity (the result is then 0);
// __fdividef returns 0 for divisors above 2^126, which is the same.  Its two
// units of the last place are as good as the exponential's, and unlike the
// exact division it has no branch, so that a lane's elements overlap.
template <bool ACCURATE>
__device__ __forceinline__ float gate_sigmoid(float x) {
    return __fdividef(1.0f, 1.0f + gate_exp<ACCURATE>(-x));
}

// act(g).  GELU's tanh form is g * sigmoid(2 c (g + k g^3)).
template <bool ACCURATE>
__device__ __forceinline__ float gate_act(float g, int act) {
    if (act == kGateSilu) return g * gate_sigmoid<ACCURATE>(g);
    if (act == kGateGelu)
        return g * gate_sigmoid<ACCURATE>(2.0f * kGeluC * fmaf(kGeluK * g * g, g, g));
    return g > 0.0f ? g : (g != g ? g : 0.0f);
}

// act(g) and act'(g).
template <bool ACCURATE>
__device__ __forceinline__ void gate_act_slope(float g, int act, float &a, float &slope) {
    if (act == kGateSilu) {
        const float s = gate_sigmoid<ACCURATE>(g);
        a = g * s;
        slope = fmaf(a, 1.0f - s, s);
    } else if (act == kGateGelu) {
        const float s = gate_sigmoid<ACCURATE>(2.0f * kGeluC * fmaf(kGeluK * g * g, g, g));
        a = g * s;
        // d/dg [g s(w)] = s + g s (1 - s) w',  w' = 2 c (1 + 3 k g^2).  From |g| = 16 on
        // s (1 - s) is zero in FP32; there w' is held at a finite value, which g^2 is
        // not above 10^19 (and zero times infinity is NaN, where the slope is 0 or 1).
        const float t = fminf(fabsf(g), 64.0f);
        slope = fmaf(a * (1.0f - s), 2.0f * kGeluC * fmaf(3.0f * kGeluK * t, t, 1.0f), s);
    } else {
        a = g > 0.0f ? g : (g != g ? g : 0.0f);
        slope = g > 0.0f ? 1.0f : 0.0f;
    }
}

}  // namespace sgemm
