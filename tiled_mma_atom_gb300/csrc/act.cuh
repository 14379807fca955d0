// act.cuh — activations of the grouped and the dense products and their
// derivatives, on one fp32 value.
//
// SiLU: silu(z) = z p, p = 1 / (1 + e^-z); silu'(z) = p (1 + z (1 - p)).
// GELU: z Phi(z), with Phi from Abramowitz & Stegun, Handbook of Mathematical
// Functions, formula 7.1.26 (|error| <= 1.5e-7 in erfc); its exponential
// e^(-z^2/2) is the one of the derivative Phi(z) + z e^(-z^2/2) / sqrt(2 pi).
// The exponential and the reciprocal are the approximate instructions (ex2 and
// rcp, a few fp32 ulp), far below the bf16 rounding of the results they enter, and
// within the fp32 sum of the bias gradient.  So is the formula but in GELU's lower
// tail, where its error is measured against a vanishing erfc: relative to the
// result 0.05 % at z = -4, 0.16 % at -5, 0.36 % at -6 (where GELU is -6e-9), 1 % at
// -8 (-5e-15), beside 0.2 to 0.4 % of a bf16 rounding.  Factors of 1/2, 1/sqrt 2 and
// log2 e are folded into the constants: 14 instructions a GELU.  With 30 (expf and
// a division) a 1024 x 4096 x 4096 product with bias, GELU and residual took 36.0
// us, against 34.8.  For z < -88 the exponential is +inf and p is 0, so silu(z)
// = -0 and not NaN.
#pragma once

#include <cuda_runtime.h>

namespace tmg {

// Values of tmg_activation.
enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActSwiglu = 4, kActSwigluGrad = 5 };

__device__ __forceinline__ float ex2_f(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_f(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid_f(float z) { return rcp_f(1.f + ex2_f(-kLog2E * z)); }

__device__ __forceinline__ float silu_f(float z) { return z * sigmoid_f(z); }

// Phi(z), and e = e^(-z^2/2).
__device__ __forceinline__ float normal_cdf(float z, float &e)
{
    const float t = rcp_f(fmaf(0.3275911f * 0.70710678118654752f, fabsf(z), 1.f));
    e = ex2_f(z * z * (-0.5f * kLog2E));
    // half of erfc(|z| / sqrt 2)
    const float half = t * e * fmaf(fmaf(fmaf(fmaf(0.5f * 1.061405429f, t, 0.5f * -1.453152027f), t, 0.5f * 1.421413741f), t,
                                         0.5f * -0.284496736f), t, 0.5f * 0.254829592f);
    return z >= 0.f ? 1.f - half : half;
}

template <int ACT>
__device__ __forceinline__ float act_f(float z)
{
    if constexpr (ACT == kActRelu)
        return z <= 0.f ? 0.f : z;          // NaN stays NaN, as fmaxf would not have it
    if constexpr (ACT == kActSilu)
        return silu_f(z);
    if constexpr (ACT == kActGelu) {
        float e;
        return z * normal_cdf(z, e);
    }
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_grad(float z)
{
    if constexpr (ACT == kActRelu)
        return z > 0.f ? 1.f : 0.f;
    if constexpr (ACT == kActSilu) {
        const float p = sigmoid_f(z);
        return p * fmaf(z, 1.f - p, 1.f);
    }
    if constexpr (ACT == kActGelu) {
        float e;
        const float c = normal_cdf(z, e);
        return fmaf(z * 0.39894228040143268f, e, c);
    }
    return 1.f;
}

// D = silu(g) u: given da = dD, the gradients of g and u.
__device__ __forceinline__ void swiglu_grad(float da, float g, float u, float &dg, float &du)
{
    const float p = sigmoid_f(g);
    du = da * g * p;
    dg = da * u * p * fmaf(g, 1.f - p, 1.f);
}

}  // namespace tmg
