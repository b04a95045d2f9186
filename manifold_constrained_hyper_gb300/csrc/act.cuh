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

// act(z). The approximate exponential is off by 2 + |z| * 1.2 ulp, which the exact one is not; every
// output is of 16 bits, or has z's own rounding of an fp32 sum beside it.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == MHC_LINEAR_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
    if (ACT == MHC_LINEAR_RELU2) return z > 0.f ? z * z : (z != z ? z : 0.f);
    if (ACT == MHC_LINEAR_SILU) return z * sigmoid_of(z);
    if (ACT == MHC_LINEAR_GELU) return 0.5f * z * erfcf(-0.70710678118654752f * z);
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
    if (ACT == MHC_LINEAR_GELU)
        return fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), 0.5f * erfcf(-0.70710678118654752f * z));
    if (ACT == MHC_LINEAR_GELU_TANH) {
        // far out, where the slope is 0 or 1, the square stays finite
        const float q = fminf(z * z, 1e8f);
        float s, t;
        sigmoid_pair(z * fmaf(kGeluB, q, kGeluA), &s, &t);
        return fmaf(z * s * t, fmaf(3.f * kGeluB, q, kGeluA), s);
    }
    return 1.f;
}
template <bool SLOPE, int ACT>
__device__ __forceinline__ float act_either(float z) {
    return SLOPE ? act_slope<ACT>(z) : act_value<ACT>(z);
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
