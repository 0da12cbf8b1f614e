// gated_math.hpp -- the gated scan's per-element mathematics, shared by its
// per-lane walk (gated.hip) and its tiled form (gated_fused.hip).
//
//   r = sigmoid(gate_r),  i = sigmoid(gate_i),  y = -scale softplus(decay) r,
//   a = e^y,  beta = sqrt(1 - a^2),  u = i x,      h_t = a_t h_{t-1} + beta_t u_t
//
// Everything is fp32 with the hardware exp2, reciprocal and square root (one
// ulp each), so a costs one exp2 and one reciprocal more than a stored
// transition would cost a load.
#pragma once

#include "device.hpp"

namespace lrscan {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2Ln2 = -0.52876637294489770f;  // log2(ln 2)

// softplus(x) = max(x, 0) + log(1 + e), e = e^-|x|, once per channel.  The
// logarithm is 2 artanh(t) with t = e / (2 + e) <= 1/3, by its series; the first
// term left out is below 2^-25 of the sum.
__device__ __forceinline__ float softplus_f(float x) {
    const float e = expf(-fabsf(x));
    const float t = e / (2.0f + e), q = t * t;
    float s = 1.0f / 13.0f;
    s = fmaf(s, q, 1.0f / 11.0f);
    s = fmaf(s, q, 1.0f / 9.0f);
    s = fmaf(s, q, 1.0f / 7.0f);
    s = fmaf(s, q, 1.0f / 5.0f);
    s = fmaf(s, q, 1.0f / 3.0f);
    s = fmaf(s * q, t, t);
    return fmaxf(x, 0.0f) + 2.0f * s;
}

// sigmoid(x) / softplus(x): the factor that takes sum P to grad_decay.  Below
// -16 the quotient is 1 - e^x / 2, which is 1 in fp32, while its numerator and
// denominator both go to zero.
__device__ __forceinline__ float decay_slope(float x) {
    return x < -16.0f ? 1.0f : 1.0f / ((1.0f + expf(-x)) * softplus_f(x));
}

// -scale softplus(decay) log2(e): y in units of log 2 is this times r.
__device__ __forceinline__ float gate_rate(float decay, float scale) {
    return -(scale * softplus_f(decay)) * kLog2e;
}

// sigmoid(x).  e^-x may overflow to infinity (x < -88); its reciprocal is then
// the 0 that the sigmoid rounds to.
__device__ __forceinline__ float sigmoid_f(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kLog2e));
}

// sigmoid(x) with its complement, 1 - sigmoid(x) = e^-x sigmoid(x), which keeps
// its digits where the sigmoid is near 1.  Below x = -88 the product is
// infinity times zero; the minimum with 1 takes the 1 there.  (It takes the 1
// for a NaN too, which the sigmoid itself still carries.)
struct Sigmoid {
    float s, c;
};
__device__ __forceinline__ Sigmoid sigmoid_pair(float x) {
    const float e = __builtin_amdgcn_exp2f(x * -kLog2e);
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    return Sigmoid{s, fminf(e * s, 1.0f)};
}

// 1 - a^2 for a = 2^y2, y2 <= 0.  Near a = 1 the difference would cancel (a
// slow channel's 1 - a^2 of 2e-4 would keep 3 digits), so there it is
// -2 a sinh(y) by the odd series of sinh, whose next term is below 2^-24 of
// the sum for |y| < 1/4; further away the difference itself loses at most
// two bits.
__device__ __forceinline__ float one_minus_sq(float a, float y2) {
    constexpr float c0 = -2.0f * kLn2;
    constexpr float c1 = c0 * kLn2 * kLn2 / 6.0f;
    constexpr float c2 = c1 * kLn2 * kLn2 / 20.0f;
    const float s = y2 * y2;
    const float near_one = (a * y2) * fmaf(s, fmaf(s, c2, c1), c0);
    return y2 > -0.36f ? near_one : fmaf(-a, a, 1.0f);
}

// The transition and the input term of one step.
struct GatedStep {
    float a, b;
};
__device__ __forceinline__ GatedStep gated_step_of(float x, float gr, float gi, float rate) {
    const float y2 = rate * sigmoid_f(gr);
    const float a = __builtin_amdgcn_exp2f(y2);
    const float beta = __builtin_amdgcn_sqrtf(one_minus_sq(a, y2));
    return GatedStep{a, beta * (sigmoid_f(gi) * x)};
}
// ... of a step that starts a segment: a = 0, beta = 1.
__device__ __forceinline__ GatedStep gated_start_of(float x, float gi) {
    return GatedStep{0.0f, sigmoid_f(gi) * x};
}

// The transition alone (the adjoint's map needs no input term).
__device__ __forceinline__ float gated_a_of(float gr, float rate) {
    return __builtin_amdgcn_exp2f(rate * sigmoid_f(gr));
}

// Gradients of one step from its adjoint lam and the state before it:
//   du = lam beta,  dx = du i,  dgi = dx x (1 - i),
//   P = y dL/dy = lam a y (h_prev - a u / beta),  dgr = P (1 - r),
// and sum P gives grad_decay (times ln 2 for a y in units of log 2).  y / beta
// is finite down to beta = 0 (y and beta^2 vanish together), so P is formed
// from a y2 and y2 / beta.  a is the transition, and p is P / ln 2 (its sum
// takes the factor once).
struct GatedGrad {
    float dx, dgr, dgi, p, a;
};
__device__ __forceinline__ GatedGrad gated_grad_of(float x, float gr, float gi, float rate,
                                                   float h_prev, float lam) {
    // r with ln 2 (1 - r): the factor comes with the exponential
    const float er = __builtin_amdgcn_exp2f(fmaf(gr, -kLog2e, kLog2Ln2));
    const float r = __builtin_amdgcn_rcpf(fmaf(er, kLog2e, 1.0f));
    const float cr = fminf(er * r, kLn2);
    const Sigmoid ig = sigmoid_pair(gi);
    const float y2 = rate * r;
    const float a = __builtin_amdgcn_exp2f(y2);
    const float v = one_minus_sq(a, y2);
    // i / beta; below 2^-126, where the reciprocal root of a denormal would be
    // infinite, beta counts as 1e-19: y / beta is near its limit 0 then anyway
    const float w = __builtin_amdgcn_rsqf(fmaxf(v, 0x1p-126f)) * ig.s;
    GatedGrad o;
    o.dx = lam * (v * w);
    o.dgi = (o.dx * x) * ig.c;
    o.p = lam * ((a * y2) * fmaf(-a, w * x, h_prev));
    o.dgr = o.p * cr;
    o.a = a;
    return o;
}
__device__ __forceinline__ GatedGrad gated_start_grad_of(float x, float gi, float lam) {
    const Sigmoid ig = sigmoid_pair(gi);
    GatedGrad o;
    o.dx = lam * ig.s;
    o.dgi = (o.dx * x) * ig.c;
    o.p = 0.0f;
    o.dgr = 0.0f;
    o.a = 0.0f;
    return o;
}

}  // namespace lrscan
