// act.cuh -- the activations of the linear products and their derivatives, in
// fp32. Each is chosen at compile time.
#pragma once

#include "common.cuh"

namespace moe {

// 2^v to 2 units in the last place, 0 below 2^-126.
__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// 1 / (1 + e^-v). The fast division returns 0 once e^-v passes 2^126, where
// the value is below 2^-126 anyway.
__device__ __forceinline__ float sigmoid_f(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// tanh form of gelu: z/2 (1 + tanh u) = z sigmoid(2u), u = sqrt(2/pi)(z + 0.044715 z^3)
__device__ __forceinline__ float gelu_tanh_2u(float z)
{
    return 1.5957691216057308f * fmaf(0.044715f * z * z, z, z);
}

// Normal distribution function:
//   Phi(-|z|) = 2^(Q(|z|) - z^2 / (2 ln 2)),
// Q the polynomial of degree 9 that fits log2 of e^{z^2/2} Phi(-|z|) over [0, 6], its error
// weighted by Phi + 0.03 (fitted for this file): 1.4e-7 of Phi's error at most, with fp32's
// roundings, and 5e-6 relative to it in the lower tail, where 1 + erf(z / sqrt 2)
// cancels. (Sums of the derivative are given in fp32: a degree of 7 left them 3e-6 off.)
// Past 6, where Phi is below 1e-9, Q stays at its end and z^2 goes on. One exponential
// and no division: the special function unit takes 8 cycles a warp, as long as 8
// multiplications.
__device__ __forceinline__ float normal_cdf(float z)
{
    const float a = fminf(fabsf(z), 6.f);
    float q = 8.469966111e-08f;
    q = fmaf(q, a, -2.2674993e-06f);
    q = fmaf(q, a, 2.335401034e-05f);
    q = fmaf(q, a, -8.848603553e-05f);
    q = fmaf(q, a, -0.0004129940448f);
    q = fmaf(q, a, 0.007469247113f);
    q = fmaf(q, a, -0.05280315618f);
    q = fmaf(q, a, 0.2622472461f);
    q = fmaf(q, a, -1.151118866f);
    q = fmaf(q, a, -0.9999997251f);
    const float h = exp2_fast(fmaf(-0.72134752f * z, z, q));
    return z > 0.f ? 1.f - h : h;
}

template <int ACT>
__device__ __forceinline__ float act_f(float z)
{
    if (ACT == MOE_ACT_RELU)
        return z > 0.f || z != z ? z : 0.f;   // NaN stays
    if (ACT == MOE_ACT_GELU)
        return z * normal_cdf(z);
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
    if (ACT == MOE_ACT_GELU)   // Phi(z) + z phi(z)
        return fmaf(0.39894228040143268f * z, exp2_fast(-0.72134752f * z * z), normal_cdf(z));
    if (ACT == MOE_ACT_GELU_TANH) {
        // d/dz [z s(v)] = s + z s (1 - s) v', v = 2u, v' = 2 sqrt(2/pi)(1 + 3 0.044715 z^2).
        // From |z| = 11 on s (1 - s) is 0 in fp32; the last factor, which leaves fp32 at 5e19,
        // is kept finite so that the product is 0 as well (a NaN comes through s).
        const float s = sigmoid_f(gelu_tanh_2u(z));
        return s + z * s * (1.f - s) * 1.5957691216057308f * fminf(fmaf(0.134145f * z, z, 1.f), 3e38f);
    }
    if (ACT == MOE_ACT_SILU) {
        const float s = sigmoid_f(z);
        return s * (1.f + z * (1.f - s));
    }
    return 1.f;
}

} // namespace moe
