// activation.hpp -- the activations of a linear layer and their slopes, in fp32.
//   relu2  max(z, 0)^2
//   silu   z p(z),  p(z) = 1 / (1 + e^-z)
//   gelu   z (1 + tanh u) / 2 = z p(2 u),  u = sqrt(2 / pi) (z + 0.044715 z^3)
// p goes by e^-|z|, which neither overflows nor cancels.
#pragma once

#include <type_traits>

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

// p(z) to 2^-23 (1 + |z|) of its value, in half the instructions: for results in
// bf16.  (e^-z may overflow: p is then 0.)
__device__ __forceinline__ float logistic_near(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
}

// kExact: to a few units of 2^-24; otherwise for a result in bf16.
template <int kAct, bool kExact>
__device__ __forceinline__ float activated(float z)
{
    if constexpr (kAct == NVFP4_ACT_RELU2) {
        const float r = z < 0.0f ? 0.0f : z;  // (keeps NaN)
        return r * r;
    } else if constexpr (kAct == NVFP4_ACT_SILU) {
        return z * (kExact ? logistic(z) : logistic_near(z));
    } else if constexpr (kAct == NVFP4_ACT_GELU) {
        const float u = kGelu * __builtin_fmaf(kGeluCube * z * z, z, z);
        return z * (kExact ? logistic(u) : logistic_near(u));
    }
    return z;
}

// The same of many values: one branch for them all.
template <bool kExact, int kCount>
__device__ __forceinline__ void activate(int act, float (&z)[kCount])
{
    const auto all = [&](auto which) {
#pragma unroll
        for (int i = 0; i < kCount; ++i) z[i] = activated<which.value, kExact>(z[i]);
    };
    if (act == NVFP4_ACT_RELU2) all(std::integral_constant<int, NVFP4_ACT_RELU2>());
    else if (act == NVFP4_ACT_SILU) all(std::integral_constant<int, NVFP4_ACT_SILU>());
    else if (act == NVFP4_ACT_GELU) all(std::integral_constant<int, NVFP4_ACT_GELU>());
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
