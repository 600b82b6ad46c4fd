// 8-bit codes of a row: q = round(127 a / top), top the row's largest magnitude
// (at least 2^-96).
//
// The codes are those of exact arithmetic.  In FP32 127 a / top is off by some
// 2^-23 of itself per operation, which decides wrongly only where it lies that near to
// the middle between two codes: such an element (some 2 in 10,000) is taken again
// in more bits, and so is the row's largest magnitude.
#pragma once

#include "ops_common.cuh"

namespace sgemm {

constexpr float kRowTiny = 0x1p-96f;

// The code of a (FP32, times inv = 127 / top), and whether |127 a / top|, off by
// at most `off`, may lie on the other side of a border.
__device__ __forceinline__ int row_code(float a, float inv, float off, bool &near) {
    const float t = a * inv;
    const float q = rintf(t);
    near = fabsf(t - q) > 0.5f - off;
    return __float2int_rn(q);
}

// round(127 a / top) in 64 bits: on which side of the middle between the codes k and
// k + 1 it lies (inv as above finds k, wherever else the quotient is near to).  What
// is in the middle but for the last bits of 64 is there exactly: an element with the same gate
// or weight as the largest, whose quotient is one of two short numbers.
__device__ __forceinline__ int row_code_exact(double a, double top, float inv) {
    const float k = floorf((float)a * inv);
    const double t = 127.0 * a, d = fma(-((double)k + 0.5), top, t);
    const int low = __float2int_rn(k);
    if (fabs(d) <= 0x1p-49 * fabs(t)) return low + (low & 1);
    return d > 0.0 ? low + 1 : low;
}

// A value as the sum of two floats, the second at most half a unit of the last
// place of the first: 48 bits.  (Sums and products without error: Knuth; Dekker.)
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_quick(float a, float b) {  // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fadd_rn(b, -__fadd_rn(s, -a))};
}
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), v = __fadd_rn(s, -a);
    return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -v)), __fadd_rn(b, -v))};
}
__device__ __forceinline__ Two two_prod(float a, float b) {
    const float p = __fmul_rn(a, b);
    return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    const Two s = two_sum(a.hi, b.hi), t = two_sum(a.lo, b.lo);
    const Two u = two_quick(s.hi, __fadd_rn(s.lo, t.hi));
    return two_quick(u.hi, __fadd_rn(u.lo, t.lo));
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
    const Two p = two_prod(a.hi, b.hi);
    return two_quick(p.hi, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, p.lo)));
}
// a / b: a quotient in FP32 and what remains, divided again.
__device__ __forceinline__ Two operator/(Two a, Two b) {
    const float q = __fdiv_rn(a.hi, b.hi);
    const Two p = Two{q, 0.0f} * b;
    const float r = __fadd_rn(__fadd_rn(__fadd_rn(a.hi, -p.hi), -p.lo), a.lo);
    return two_quick(q, __fdiv_rn(r, b.hi));
}

// exp(-x) for x in [0, 60]: x = n ln 2 + r, Taylor's series of exp(-r) for |r| <= ln 2 / 2
// to the 12th power (remainder 2^-52 of the sum), the powers from the 7th on in FP32
// (together below 2^-22 of the sum, so their rounding is below 2^-46).
static __device__ __noinline__ Two two_exp_neg(Two x) {
    const float n = rintf(x.hi * 1.4426950408889634f);
    // ln 2 in three parts; the first has 12 bits, so that n times it is exact.
    constexpr double kLn2 = 0.693147180559945309417;
    constexpr float l1 = 2839.0f / 4096.0f;
    constexpr float l2 = (float)(kLn2 - l1);
    constexpr float l3 = (float)(kLn2 - l1 - l2);
    const Two n2 = two_prod(-n, l2);
    Two r = two_sum(__fmaf_rn(-n, l1, x.hi), n2.hi);
    r = r + Two{__fadd_rn(x.lo, n2.lo), 0.0f};
    r = r + Two{-n * l3, 0.0f};
    r = Two{-r.hi, -r.lo};
    // 1/12! ... 1/7!
    float tail = 2.08767569878681e-09f;
    tail = fmaf(tail, r.hi, 2.505210838544172e-08f);
    tail = fmaf(tail, r.hi, 2.755731922398589e-07f);
    tail = fmaf(tail, r.hi, 2.755731922398589e-06f);
    tail = fmaf(tail, r.hi, 2.48015873015873e-05f);
    tail = fmaf(tail, r.hi, 1.984126984126984e-04f);
    Two e = Two{tail, 0.0f} * r;
    constexpr double c6 = 1.0 / 720, c5 = 1.0 / 120, c4 = 1.0 / 24, c3 = 1.0 / 6;
    e = e + Two{(float)c6, (float)(c6 - (float)c6)};
    e = e * r + Two{(float)c5, (float)(c5 - (float)c5)};
    e = e * r + Two{(float)c4, (float)(c4 - (float)c4)};
    e = e * r + Two{(float)c3, (float)(c3 - (float)c3)};
    e = e * r + Two{0.5f, 0.0f};
    e = e * r + Two{1.0f, 0.0f};
    e = e * r + Two{1.0f, 0.0f};
    const float scale = __int_as_float((127 - (int)n) << 23);  // 2^-n, n <= 87
    return Two{e.hi * scale, e.lo * scale};
}

}  // namespace sgemm
