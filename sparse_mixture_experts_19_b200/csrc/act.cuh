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

// Phi(z), the normal distribution function, and e^(-z^2/2): with x = |z| / sqrt 2
// and t = 1 / (1 + 0.3275911 x), erfc(x) = (a1 t + ... + a5 t^5) e^(-x^2) to within
// 1.5e-7 (Abramowitz and Stegun, formula 7.1.26), a fifth of erfcf's time in a
// matrix product's epilogue (10 us of a 30 us call).  In the lower tail Phi is
// this product itself, not one minus it, so it falls off to zero as it should.
__device__ __forceinline__ float normal_cdf_f32(float z, float& gauss) {
    const float t = rcp_f32(fmaf(0.23164189f, fabsf(z), 1.f));
    gauss = exp2_f32(-0.5f * kLog2e * z * z);
    float p = fmaf(1.061405429f, t, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f);
    const float q = 0.5f * p * t * gauss;
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
