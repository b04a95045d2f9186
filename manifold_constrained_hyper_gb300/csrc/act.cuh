// The activations of a product's epilogue and their slopes, in fp32.
#pragma once
#include <type_traits>

#include "block_common.cuh"

namespace mhc {

// 1 / (1 + exp(-z)) without overflow, the divisor in [1, 2], where the approximate division is off by 2 ulp.
__device__ __forceinline__ float sigmoid_of(float z) {
    const float e = __expf(-fabsf(z));
    return __fdividef(z < 0.f ? e : 1.f, 1.f + e);
}
// It and what it lacks to 1, neither by cancellation.
__device__ __forceinline__ void sigmoid_pair(float z, float *s, float *t) {
    const float e = __expf(-fabsf(z)), r = __fdividef(1.f, 1.f + e);
    *s = z < 0.f ? e * r : r;
    *t = z < 0.f ? r : e * r;
}
// gelu's tanh form is z * sigmoid(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3): no cancellation far below zero.
constexpr float kGeluA = 1.5957691216057308f, kGeluB = 0.07135481627260025f;   // 2 sqrt(2/pi), and 0.044715 of it

// What the normal distribution has beyond |z|, E = exp(-z^2 / 2) given: erfc(|z| / sqrt 2) / 2 = E t P(t) with t = 1 / (1 +
// 0.4 |z| / sqrt 2). P fits exp(x^2) erfc(x) / t to 1.3e-7 of itself for all x >= 0 (least squares on 6000 Chebyshev points, weighted
// until the largest relative errors are level); 5e-7 in fp32. Some 15 instructions, a third of erfcf's.
__device__ __forceinline__ float normal_tail(float z, float E) {
    const float t = __fdividef(1.f, fmaf(0.28284271247461903f, fabsf(z), 1.f));
    float p = 0.05025513097643852f * 0.5f;
    p = fmaf(p, t, -0.18287666141986847f * 0.5f);
    p = fmaf(p, t, 0.16905011236667633f * 0.5f);
    p = fmaf(p, t, -0.005581708624958992f * 0.5f);
    p = fmaf(p, t, 0.1414211392402649f * 0.5f);
    p = fmaf(p, t, 0.16854415833950043f * 0.5f);
    p = fmaf(p, t, 0.20784246921539307f * 0.5f);
    p = fmaf(p, t, 0.22566960752010345f * 0.5f);
    p = fmaf(p, t, 0.22567586600780487f * 0.5f);
    return p * t * E;
}
// act(z). The approximate exponential is off by 2 + |z| * 1.2 ulp, which the exact one is not; every
// output is of 16 bits, or has z's own rounding of an fp32 sum beside it.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == MHC_LINEAR_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
    if (ACT == MHC_LINEAR_RELU2) return z > 0.f ? z * z : (z != z ? z : 0.f);
    if (ACT == MHC_LINEAR_SILU) return z * sigmoid_of(z);
    if (ACT == MHC_LINEAR_GELU) {
        const float q = normal_tail(z, __expf(-0.5f * z * z));
        return z * (z < 0.f ? q : 1.f - q);
    }
    if (ACT == MHC_LINEAR_GELU_TANH) return z * sigmoid_of(z * fmaf(kGeluB, z * z, kGeluA));
    return z;
}
// act'(z)
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if (ACT == MHC_LINEAR_RELU) return z > 0.f ? 1.f : (z != z ? z : 0.f);
    if (ACT == MHC_LINEAR_RELU2) return z > 0.f ? 2.f * z : (z != z ? z : 0.f);
    if (ACT == MHC_LINEAR_SILU) {
        float s, t;
        sigmoid_pair(z, &s, &t);
        return fmaf(z * s, t, s);
    }
    if (ACT == MHC_LINEAR_GELU) {
        // far out, where the slope is 0 or 1, z times 0 stays finite
        const float E = __expf(-0.5f * z * z), q = normal_tail(z, E);
        return fmaf(z * 0.39894228040143268f, E, z < 0.f ? q : 1.f - q);
    }
    if (ACT == MHC_LINEAR_GELU_TANH) {
        // far out, where the slope is 0 or 1, the square stays finite
        const float q = fminf(z * z, 1e8f);
        float s, t;
        sigmoid_pair(z * fmaf(kGeluB, q, kGeluA), &s, &t);
        return fmaf(z * s * t, fmaf(3.f * kGeluB, q, kGeluA), s);
    }
    return 1.f;
}
// f(an integral constant of the activation), the switch outside of what f loops over.
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
    switch (act) {
    case MHC_LINEAR_RELU: f(std::integral_constant<int, MHC_LINEAR_RELU>()); break;
    case MHC_LINEAR_RELU2: f(std::integral_constant<int, MHC_LINEAR_RELU2>()); break;
    case MHC_LINEAR_SILU: f(std::integral_constant<int, MHC_LINEAR_SILU>()); break;
    case MHC_LINEAR_GELU: f(std::integral_constant<int, MHC_LINEAR_GELU>()); break;
    case MHC_LINEAR_GELU_TANH: f(std::integral_constant<int, MHC_LINEAR_GELU_TANH>()); break;
    default: f(std::integral_constant<int, MHC_LINEAR_NONE>()); break;
    }
}

}  // namespace mhc
