// activation.hpp -- the activations of a linear layer and their slopes, in fp32.
//   relu2  max(z, 0)^2
//   silu   z p(z),  p(z) = 1 / (1 + e^-z)
//   gelu   z (1 + tanh u) / 2 = z p(2 u),  u = sqrt(2 / pi) (z + 0.044715 z^3)
// p goes by e^-|z|, which neither overflows nor cancels.
#pragma once

#include "nvfp4.h"
#include "wave.hpp"

namespace nvfp4 {

__device__ __forceinline__ float logistic(float z)
{
    const float e = exp_neg(-__builtin_fabsf(z));
    return (z < 0.0f ? e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + e);
}

constexpr float kGelu = 1.5957691216f;  // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

__device__ __forceinline__ float activation(int act, float z)
{
    if (act == NVFP4_ACT_RELU2) {
        const float r = z < 0.0f ? 0.0f : z;  // (keeps NaN)
        return r * r;
    }
    if (act == NVFP4_ACT_SILU) return z * logistic(z);
    if (act == NVFP4_ACT_GELU) return z * logistic(kGelu * __builtin_fmaf(kGeluCube * z * z, z, z));
    return z;
}

__device__ __forceinline__ float activation_slope(int act, float z)
{
    if (act == NVFP4_ACT_RELU2) return z < 0.0f ? 0.0f : 2.0f * z;
    if (act == NVFP4_ACT_SILU) {
        const float p = logistic(z);
        return p * __builtin_fmaf(z, 1.0f - p, 1.0f);
    }
    if (act == NVFP4_ACT_GELU) {
        // beyond 64 p is 0 or 1, and the cubic would overflow
        const float x = z > 64.0f ? 64.0f : z < -64.0f ? -64.0f : z, square = x * x;
        const float p = logistic(kGelu * __builtin_fmaf(kGeluCube * square, x, x));
        return __builtin_fmaf(x * p * (1.0f - p), kGelu * __builtin_fmaf(3.0f * kGeluCube, square, 1.0f), p);
    }
    return 1.0f;
}

}  // namespace nvfp4
