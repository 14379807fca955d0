// act.cuh — activations of the grouped and the dense products and their
// derivatives, on one fp32 value.
//
// SiLU: silu(z) = z p, p = 1 / (1 + e^-z); silu'(z) = p (1 + z (1 - p)).
// GELU: z Phi(z), with Phi from Abramowitz & Stegun, Handbook of Mathematical
// Functions, formula 7.1.26 (|error| <= 1.5e-7 in erfc); its exponential
// e^(-z^2/2) is the one of the derivative Phi(z) + z e^(-z^2/2) / sqrt(2 pi).
// The exponential and the division are the fast intrinsics: a few fp32 ulp,
// far below the bf16 rounding of every result they enter, and within the
// fp32 sum of the bias gradient.  For z < -88 the exponential is +inf and p
// is 0 (the intrinsic division by a value above 2^126 returns 0), so
// silu(z) = -0 and not NaN.
#pragma once

#include <cuda_runtime.h>

namespace tmg {

// Values of tmg_activation.
enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActSwiglu = 4, kActSwigluGrad = 5 };

__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

__device__ __forceinline__ float silu_f(float z) { return __fdividef(z, 1.f + __expf(-z)); }

// Phi(z), and e = e^(-z^2/2).
__device__ __forceinline__ float normal_cdf(float z, float &e)
{
    const float x = fabsf(z) * 0.70710678118654752f;
    const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
    const float poly = t * fmaf(fmaf(fmaf(fmaf(1.061405429f, t, -1.453152027f), t, 1.421413741f), t, -0.284496736f), t,
                                0.254829592f);
    e = __expf(-x * x);
    const float half = 0.5f * poly * e;
    return z >= 0.f ? 1.f - half : half;
}

template <int ACT>
__device__ __forceinline__ float act_f(float z)
{
    if constexpr (ACT == kActRelu)
        return fmaxf(z, 0.f);
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
