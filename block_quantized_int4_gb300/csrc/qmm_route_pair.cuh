// qmm_route_pair.cuh -- router scores as unevaluated sums of two fp32 numbers
// (about 2^-42 of the largest score), for the tokens that fp32 does not order:
// the 64-bit pipe of the device takes a warp 16 cycles an instruction.
//
// Sums and products of pairs are Knuth's and Dekker's (the latter with fused
// multiply-add).  exp(x) = 2^n exp(r), r = x - n ln 2 with ln 2 in three parts of
// 15, 15 and 24 bits (n times the first two is exact); exp(r) - 1 from the Taylor
// polynomial of r / 8 (degree 7: 2^-51) and three times (1 + p)^2 - 1 = 2 p + p^2.
#pragma once

#ifdef __CUDACC__
#define QMM_PAIR __device__ __forceinline__
#else  // for a check of the arithmetic on the host
#include <math.h>
#define QMM_PAIR static inline
QMM_PAIR float __fadd_rn(float a, float b) { return a + b; }
QMM_PAIR float __fmul_rn(float a, float b) { return a * b; }
QMM_PAIR float __fmaf_rn(float a, float b, float c) { return fmaf(a, b, c); }
#endif

namespace qmm {
namespace route {

struct Pair {
    float hi, lo;  // |lo| at most half a step of hi
};

QMM_PAIR Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
    return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t))};
}
QMM_PAIR Pair quick_sum(float a, float b) {  // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fadd_rn(b, -__fadd_rn(s, -a))};
}
QMM_PAIR Pair add(Pair a, Pair b) {
    const Pair s = two_sum(a.hi, b.hi), t = two_sum(a.lo, b.lo);
    const Pair u = quick_sum(s.hi, __fadd_rn(s.lo, t.hi));
    return quick_sum(u.hi, __fadd_rn(u.lo, t.lo));
}
QMM_PAIR Pair add(Pair a, float b) {
    const Pair s = two_sum(a.hi, b);
    return quick_sum(s.hi, __fadd_rn(s.lo, a.lo));
}
QMM_PAIR Pair mul(Pair a, Pair b) {
    const float p = __fmul_rn(a.hi, b.hi);
    const float e = __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.hi, -p)));
    return quick_sum(p, e);
}
QMM_PAIR Pair scaled(Pair a, float power_of_two) {
    return {__fmul_rn(a.hi, power_of_two), __fmul_rn(a.lo, power_of_two)};
}

// exp(x) for |x| <= 87.
QMM_PAIR Pair exp_pair(Pair x) {
    const float n = rintf(__fmul_rn(x.hi, 1.4426950408889634f));
    Pair r = two_sum(__fmaf_rn(n, -0x1.62e4p-1f, x.hi), __fmul_rn(n, -0x1.7f7cp-20f));
    r = quick_sum(r.hi, __fadd_rn(r.lo, __fmaf_rn(n, -0x1.1cf79ap-36f, x.lo)));
    const Pair s = scaled(r, 0.125f), s2 = mul(s, s);
    const Pair s3 = mul(mul(s2, s), Pair{0x1.555556p-3f, -0x1.555556p-28f});  // s^3 / 6
    const float s4 = __fmul_rn(s2.hi, s2.hi), h = s.hi;
    const float rest = __fmul_rn(s4, __fmaf_rn(h, __fmaf_rn(h, __fmaf_rn(h, 1.f / 5040.f, 1.f / 720.f), 1.f / 120.f),
                                               1.f / 24.f));
    Pair p = add(s, add(scaled(s2, 0.5f), add(s3, rest)));
    p = add(scaled(p, 2.f), mul(p, p));
    p = add(scaled(p, 2.f), mul(p, p));
    p = add(scaled(p, 2.f), mul(p, p));
    p = add(p, 1.f);
    const float half = ldexpf(1.f, (int)n / 2), other = ldexpf(1.f, (int)n - (int)n / 2);
    return scaled(scaled(p, half), other);
}

// 1 / x for x >= 2^-100, about.
QMM_PAIR Pair reciprocal(Pair x) {
    const float r = 1.f / x.hi;
    const float e = __fmaf_rn(-x.lo, r, __fmaf_rn(-x.hi, r, 1.f));
    return quick_sum(r, __fmul_rn(r, __fmaf_rn(e, e, e)));
}

QMM_PAIR Pair sigmoid_pair(float l) {
    const float x = l > 87.f ? -87.f : l < -87.f ? 87.f : -l;
    return reciprocal(add(exp_pair(Pair{x, 0.f}), 1.f));
}

QMM_PAIR bool before(Pair a, Pair b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }

// Whether two values may be in either order when their difference is off by up to
// `tolerance`.  What takes no part (-inf) is last, however large the tolerance.
QMM_PAIR bool unsure(Pair a, Pair b, float tolerance) {
    const float d = fabsf(__fadd_rn(__fadd_rn(a.hi, -b.hi), __fadd_rn(a.lo, -b.lo)));
    return a.hi > -INFINITY && b.hi > -INFINITY && d <= tolerance;
}

}  // namespace route
}  // namespace qmm
