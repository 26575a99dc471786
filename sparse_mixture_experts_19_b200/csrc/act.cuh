// Activations of the gate/up projections and the linear layer, float32.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace moe {

// The special function unit's 2^x and 1/x (2 and 1 units in the last place), with
// results below the normal range as 0: the forms that keep those take three
// instructions more each (GELU forward, 8191 x 2880 -> 2880: 109.9 us with those,
// 106.3 with these).
__device__ __forceinline__ float exp2_f32(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_f32(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// p(z) = 1 / (1 + e^-z): an infinite e^-z gives 0.
__device__ __forceinline__ float sigmoid_f32(float z) { return rcp_f32(1.f + exp2_f32(-kLog2e * z)); }

// sqrt(2 / pi) (z + 0.044715 z^3), doubled: tanh-form GELU is z sigmoid(this).
__device__ __forceinline__ float gelu_tanh_arg(float z) {
    return 1.5957691216057308f * fmaf(0.044715f * z * z, z, z);
}

// Phi(z), the normal distribution function, and e^(-z^2/2): with x = |z| and
// t = 1 / (1 + 0.29 x), Phi(-x) = t P(t) e^(-x^2/2), P of degree 5.  P was fitted
// to erfcx(x / sqrt 2) / 2 (a linear program for the least largest error on 0 <= x
// <= 14) with an absolute bound near 0 and a relative one in the lower tail, so that
// this falls off to zero in step with Phi: in float32 2.4e-7 absolute, and 6e-5 of
// the value (a bf16 result's half step is 4e-3) down to z = -12.9, where z Phi(z)
// leaves the normal range.  A form with an absolute bound alone, formula 7.1.26 of
// Abramowitz and Stegun, takes as long and is 1% off at -8; degree 6 would be right
// to 1e-5 and takes 1 to 3% more of a call (dz of 8191 x 2880: 34.7 us, 33.6 with
// this).  erfcf takes five times as long in a matrix product's epilogue (10 us more
// in a 30 us call).
__device__ __forceinline__ float normal_cdf_f32(float z, float& gauss) {
    const float t = rcp_f32(fmaf(0.29f, fabsf(z), 1.f));
    gauss = exp2_f32(-0.5f * kLog2e * z * z);
    float p = fmaf(-0.0874850452f, t, 0.280140132f);
    p = fmaf(p, t, -0.0866808817f);
    p = fmaf(p, t, 0.175283223f);
    p = fmaf(p, t, 0.102007858f);
    p = fmaf(p, t, 0.116734825f);
    const float q = p * t * gauss;
    return z < 0.f ? q : 1.f - q;
}

// act(z).  ReLU keeps a NaN.
template <int kAct>
__device__ __forceinline__ float act_value(float z) {
    if (kAct == MOE_ACT_SILU) return z * sigmoid_f32(z);
    if (kAct == MOE_ACT_GELU) {
        float gauss;
        return z * normal_cdf_f32(z, gauss);
    }
    if (kAct == MOE_ACT_GELU_TANH) return z * sigmoid_f32(gelu_tanh_arg(z));
    if (kAct == MOE_ACT_RELU) return z < 0.f ? 0.f : z;
    return z;
}

// act(z) and act'(z).  The slope of the tanh form is p + z p (1 - p) q' with q'
// quadratic in z: beyond |z| = 30, where p (1 - p) is 0, z is clamped so that
// no 0 * inf arises.
template <int kAct>
__device__ __forceinline__ void act_slope(float z, float& a, float& d) {
    if (kAct == MOE_ACT_SILU) {
        const float p = sigmoid_f32(z);
        a = z * p;
        d = p * fmaf(z, 1.f - p, 1.f);
    } else if (kAct == MOE_ACT_GELU) {
        float gauss;
        const float c = normal_cdf_f32(z, gauss);
        a = z * c;
        d = fmaf(z, 0.3989422804014327f * gauss, c);
    } else if (kAct == MOE_ACT_GELU_TANH) {
        const float p = sigmoid_f32(gelu_tanh_arg(z));
        const float c = fminf(fmaxf(z, -30.f), 30.f);
        a = z * p;
        d = fmaf(c * p * (1.f - p), 1.5957691216057308f * fmaf(0.134145f * c, c, 1.f), p);
    } else if (kAct == MOE_ACT_RELU) {
        a = z < 0.f ? 0.f : z;
        d = z > 0.f ? 1.f : 0.f;
    } else {
        a = z;
        d = 1.f;
    }
}

// f(std::integral_constant<int, act>) for a run-time activation (a uniform branch).
template <typename F>
__host__ __device__ __forceinline__ void by_act(int act, F f) {
    switch (act) {
        case MOE_ACT_SILU: f(std::integral_constant<int, MOE_ACT_SILU>()); break;
        case MOE_ACT_GELU: f(std::integral_constant<int, MOE_ACT_GELU>()); break;
        case MOE_ACT_GELU_TANH: f(std::integral_constant<int, MOE_ACT_GELU_TANH>()); break;
        case MOE_ACT_RELU: f(std::integral_constant<int, MOE_ACT_RELU>()); break;
        default: f(std::integral_constant<int, MOE_ACT_NONE>()); break;
    }
}

}  // namespace moe
