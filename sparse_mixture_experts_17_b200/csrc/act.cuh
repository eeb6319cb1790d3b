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

template <int ACT>
__device__ __forceinline__ float act_f(float z)
{
    if (ACT == MOE_ACT_RELU)
        return z > 0.f || z != z ? z : 0.f;   // NaN stays
    if (ACT == MOE_ACT_GELU)
        return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
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
        return 0.5f * (1.f + erff(z * 0.70710678118654752f)) +
               z * __expf(-0.5f * z * z) * 0.39894228040143268f;
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
