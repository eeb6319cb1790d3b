// act.cuh -- the activations of the linear products and their derivatives, in
// fp32. Each is chosen at compile time.
#pragma once

#include "common.cuh"

namespace moe {

// 1 / (1 + e^-v). The fast division returns 0 once e^-v passes 2^126, where
// the value is below 2^-126 anyway.
__device__ __forceinline__ float sigmoid_f(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// tanh form of gelu: z/2 (1 + tanh u) = z sigmoid(2u), u = sqrt(2/pi)(z + 0.044715 z^3)
__device__ __forceinline__ float gelu_tanh_2u(float z)
{
    return 1.5957691216057308f * fmaf(0.044715f * z * z, z, z);
}

// Normal distribution function, and e = exp(-z^2 / 2), which its density shares:
//   Phi(-|z|) = e t q(t),  t = 1 / (1 + 0.36 |z|),
// q the polynomial of degree 6 that fits e^{z^2/2} Phi(-|z|) / t over [0, 14] with the
// least relative error, 9e-7 (fitted for this file). The relative error holds in the
// lower tail too, where 1 + erf(z / sqrt 2) cancels, and it takes 14 instructions
// where erff and an exponential of their own take about 40.
__device__ __forceinline__ float normal_cdf(float z, float &e)
{
    e = __expf(-0.5f * z * z);
    const float t = __fdividef(1.f, fmaf(0.36f, fabsf(z), 1.f));
    float q = 0.04705785960f;
    q = fmaf(q, t, -0.1797699630f);
    q = fmaf(q, t, 0.1809608639f);
    q = fmaf(q, t, 0.02654494531f);
    q = fmaf(q, t, 0.1397207230f);
    q = fmaf(q, t, 0.1417722116f);
    q = fmaf(q, t, 0.1437130570f);
    const float h = e * t * q;
    return z > 0.f ? 1.f - h : h;
}

template <int ACT>
__device__ __forceinline__ float act_f(float z)
{
    if (ACT == MOE_ACT_RELU)
        return z > 0.f || z != z ? z : 0.f;   // NaN stays
    if (ACT == MOE_ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
    }
    if (ACT == MOE_ACT_GELU_TANH)
        return z * sigmoid_f(gelu_tanh_2u(z));
    if (ACT == MOE_ACT_SILU)
        return z * sigmoid_f(z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_grad_f(float z)
{
    if (ACT == MOE_ACT_RELU)
        return z > 0.f ? 1.f : 0.f;
    if (ACT == MOE_ACT_GELU) {   // Phi(z) + z phi(z)
        float e;
        const float phi = normal_cdf(z, e);
        return fmaf(0.39894228040143268f * z, e, phi);
    }
    if (ACT == MOE_ACT_GELU_TANH) {
        // d/dz [z s(v)] = s + z s (1 - s) v', v = 2u, v' = 2 sqrt(2/pi)(1 + 3 0.044715 z^2)
        const float s = sigmoid_f(gelu_tanh_2u(z));
        return s + z * s * (1.f - s) * 1.5957691216057308f * fmaf(0.134145f * z, z, 1.f);
    }
    if (ACT == MOE_ACT_SILU) {
        const float s = sigmoid_f(z);
        return s * (1.f + z * (1.f - s));
    }
    return 1.f;
}

} // namespace moe
