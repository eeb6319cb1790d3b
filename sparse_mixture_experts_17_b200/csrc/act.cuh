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
//   Phi(-|z|) = 2^(Q(|z|) - z^2 / (2 ln 2)).
// Up to 6, Q is the polynomial of degree 9 that fits log2 of e^{z^2/2} Phi(-|z|), its error
// weighted by Phi + 0.03 (fitted for this file). With fp32's roundings, and an exact
// exponential, Phi is off by 1.8e-7 at most (1.5e-7 for z < 0; for z > 0 the rounding of
// 1 - h is in it), and by 5.4e-6 of itself in the lower tail, where 1 + erf(z / sqrt 2)
// cancels. (Sums of the derivative are given in fp32: a degree of 7 left them 3e-6 off.)
// Past 6, where Phi is below 1e-9, a cubic in |z| - 6 continues Q: 6.6e-4 of Phi at most,
// a sixth of bf16's half step. (Q held at its end made Phi 4% too large at -6.25, 34%
// at -8.) Phi below 2^-126 (z < -12.95) counts as 0. One exponential and no division: the
// special function unit takes 8 cycles a warp, as long as 8 multiplications.
__device__ __forceinline__ float normal_q(float a)   // Q on [0, 6]
{
    float q = 8.469966111e-08f;
    q = fmaf(q, a, -2.2674993e-06f);
    q = fmaf(q, a, 2.335401034e-05f);
    q = fmaf(q, a, -8.848603553e-05f);
    q = fmaf(q, a, -0.0004129940448f);
    q = fmaf(q, a, 0.007469247113f);
    q = fmaf(q, a, -0.05280315618f);
    q = fmaf(q, a, 0.2622472461f);
    q = fmaf(q, a, -1.151118866f);
    return fmaf(q, a, -0.9999997251f);
}

// Q past 6, t = |z| - 6 (0 adds nothing). The leading coefficient is negative, so far out
// Q goes to -inf and Phi to 0.
__device__ __forceinline__ float normal_q_tail(float t, float q)
{
    return fmaf(t, fmaf(t, fmaf(t, -0.00057606207f, 0.014062471f), -0.22552708f), q);
}

__device__ __forceinline__ float normal_cdf_of(float z, float q)
{
    const float h = exp2_fast(fmaf(-0.72134752f * z, z, q));
    return z > 0.f ? 1.f - h : h;
}

// Every activation but gelu, which goes by normal_cdf_n.
template <int ACT>
__device__ __forceinline__ float act_f(float z)
{
    if (ACT == MOE_ACT_RELU)
        return z > 0.f || z != z ? z : 0.f;   // NaN stays
    if (ACT == MOE_ACT_GELU_TANH)
        return z * sigmoid_f(gelu_tanh_2u(z));
    if (ACT == MOE_ACT_SILU)
        return z * sigmoid_f(z);
    return z;
}

// Phi of N values. Values past 6 are rare, so the tail is passed by where none of the N is
// there (the same bits either way). y = gelu(16384 x 256 -> 4096), us: 83 with N = 4 or 8, 86
// with 2, 87 with the tail's four operations for every value, 79 without a tail; dz of 4096 x
// 4096 with the bias sums: 24.7 with N = 4, 25.1 with 2 or 8 (which spills), 23.5 without.
template <int N>
__device__ __forceinline__ void normal_cdf_n(const float (&z)[N], float (&phi)[N])
{
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        top = fmaxf(top, fabsf(z[i]));
        phi[i] = normal_q(fminf(fabsf(z[i]), 6.f));
    }
    if (top > 6.f) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            phi[i] = normal_q_tail(fabsf(z[i]) - fminf(fabsf(z[i]), 6.f), phi[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        phi[i] = normal_cdf_of(z[i], phi[i]);
}

// act of N values in place.
template <int ACT, int N>
__device__ __forceinline__ void act_n(float (&v)[N])
{
    float phi[N];
    if (ACT == MOE_ACT_GELU)
        normal_cdf_n(v, phi);
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = ACT == MOE_ACT_GELU ? v[i] * phi[i] : act_f<ACT>(v[i]);
}

template <int ACT>
__device__ __forceinline__ float act_grad_f(float z)
{
    if (ACT == MOE_ACT_RELU)
        return z > 0.f ? 1.f : 0.f;
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

// act' of N values in place.
template <int ACT, int N>
__device__ __forceinline__ void act_grad_n(float (&v)[N])
{
    float phi[N];
    if (ACT == MOE_ACT_GELU)   // Phi(z) + z phi(z)
        normal_cdf_n(v, phi);
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = ACT == MOE_ACT_GELU
                   ? fmaf(0.39894228040143268f * v[i], exp2_fast(-0.72134752f * v[i] * v[i]), phi[i])
                   : act_grad_f<ACT>(v[i]);
}

} // namespace moe
