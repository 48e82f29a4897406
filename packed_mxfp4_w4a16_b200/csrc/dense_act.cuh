// dense_act.cuh — activations of the gated block and their derivatives, FP32.
#pragma once

#include <cuda_runtime.h>
#include <math.h>

#include "../../include/moe_mxfp4.h"

namespace moe {

constexpr float kGeluC0 = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluC1 = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// 1 / (1 + exp(-z)), by the hardware's 2^x and reciprocal (a few 2^-23
// relative for |z| of order 1, |z| 2^-23 in the left tail: far below the
// 2^-8 of the BF16 results).  Below the same of 2 z serves the tanh form of
// GELU: (1 + tanh z) / 2 = sigmoid(2 z), which keeps the relative precision
// of the left tail where 1 + tanh z cancels.
__device__ __forceinline__ float sigmoid_f32(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// Phi(g), the normal distribution function, and e = exp(-g^2 / 2), which its
// derivative needs too.  With x = |g| / sqrt(2), Phi(-|g|) = erfc(x) / 2 and
// erfc(x) exp(x^2) is smooth: t Q(t), t = 1 / (1 + x / 2), Q of degree 8
// fitted here by weighted least squares with the weights moved to the largest
// errors (Lawson's iteration): 5e-8 relative over x in [0, 13], 1.6e-7 as
// evaluated in FP32; beyond, exp(-x^2) is 0.  Both tails keep their relative
// precision.  (erfcf took longer than the products of a short K.)
__device__ __forceinline__ float normal_cdf(float g, float &e) {
    e = __expf(-0.5f * g * g);
    const float t = __fdividef(1.0f, fmaf(0.5f * kSqrtHalf, fabsf(g), 1.0f));
    float q = -0.0593861863f;
    q = fmaf(q, t, 0.28612271f);
    q = fmaf(q, t, -0.49040401f);
    q = fmaf(q, t, 0.28173086f);
    q = fmaf(q, t, -0.029147055f);
    q = fmaf(q, t, 0.203751996f);
    q = fmaf(q, t, 0.242835224f);
    q = fmaf(q, t, 0.282412082f);
    q = fmaf(q, t, 0.282084346f);
    const float h = 0.5f * t * q * e;
    return g < 0.f ? h : 1.0f - h;
}

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
    if (ACT == MOE_ACT_SILU) return g * sigmoid_f32(g);
    if (ACT == MOE_ACT_GELU) {
        float e;
        return g * normal_cdf(g, e);
    }
    return g * sigmoid_f32(2.0f * kGeluC0 * (g + kGeluC1 * g * g * g));
}

// act(g) and act'(g).  Where the sigmoid has reached 0 or 1 its slope is 0
// whatever the factor beside it (which may have overflowed).
template <int ACT>
__device__ __forceinline__ void act_value_grad(float g, float &a, float &da) {
    if (ACT == MOE_ACT_SILU) {
        const float s = sigmoid_f32(g), t = s * (1.0f - s);
        a = g * s;
        da = s + (t > 0.f ? g * t : 0.f);
    } else if (ACT == MOE_ACT_GELU) {
        float e;
        const float cdf = normal_cdf(g, e);
        a = g * cdf;
        da = cdf + (e > 0.f ? g * (kInvSqrt2Pi * e) : 0.f);
    } else {
        const float s = sigmoid_f32(2.0f * kGeluC0 * (g + kGeluC1 * g * g * g));
        const float t = s * (1.0f - s);
        a = g * s;
        da = s + (t > 0.f ? g * t * (2.0f * kGeluC0 * (1.0f + 3.0f * kGeluC1 * g * g)) : 0.f);
    }
}

}  // namespace moe
