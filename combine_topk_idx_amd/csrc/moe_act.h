// Activations of the bf16 expert layer and their slopes, on the device.
#pragma once

#include <type_traits>

#include "moe_mma.h"
#include "moe_train_internal.h"

namespace moe {
namespace dev {

// v within +-1e6, NaN kept: past it gelu is 0 or v and its slope 0 or 1, and the cube
// would overflow.
__device__ __forceinline__ float near(float v) { return v > 1e6f ? 1e6f : v < -1e6f ? -1e6f : v; }

// gelu(v) = v / 2 (1 + tanh(z / 2)) = v / (1 + exp(-z)), z = sqrt(8/pi) (v + 0.044715 v^3)
constexpr float kGeluLinear = 1.5957691216057308f, kGeluCubic = 1.5957691216057308f * 0.044715f;
__device__ __forceinline__ float gelu_z(float v) { return v * (kGeluLinear + kGeluCubic * v * v); }

// 1 / (1 + exp(-z)) from the hardware's exp2 and reciprocal (1 step each): the
// argument's rounding costs |z| 2^-24 of exp(-z), which s (1 - s) damps to less than
// 2^-24 of 1 where s matters beside 1, and |z| 2^-24 < 2^-17 of s itself where it
// does not: far below bf16's half step of 2^-8.  The reciprocal has no subnormal
// results: s is 0 where it is below 2^-126, z < -87.3.
__device__ __forceinline__ float sigmoid(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

template <int ACT>
__device__ __forceinline__ float act_value(float v)
{
    if constexpr (ACT == MOE_ACT_SILU)
        return v * sigmoid(v);
    if constexpr (ACT == MOE_ACT_GELU)
        return v * sigmoid(gelu_z(near(v)));
    if constexpr (ACT == MOE_ACT_RELU)
        return v < 0.0f ? 0.0f : v;
    return v;
}

// The value f and the slope d of an activation at v.
template <int ACT>
__device__ __forceinline__ void act_both(float v, float &f, float &d)
{
    if constexpr (ACT == MOE_ACT_SILU) {
        const float s = sigmoid(v);
        f = v * s;
        d = s + f * (1.0f - s);
    } else if constexpr (ACT == MOE_ACT_GELU) {
        const float c = near(v);
        const float s = sigmoid(gelu_z(c));
        f = v * s;
        d = s + c * s * (1.0f - s) * (kGeluLinear + 3.0f * kGeluCubic * c * c);
    } else if constexpr (ACT == MOE_ACT_RELU) {
        f = v < 0.0f ? 0.0f : v;
        d = v <= 0.0f ? 0.0f : v > 0.0f ? 1.0f : v;
    } else {
        f = v;
        d = 1.0f;
    }
}

// f with the activation as a type.
template <typename F>
__device__ __forceinline__ void for_act(int act, const F &f)
{
    if (act == MOE_ACT_SILU)
        f(std::integral_constant<int, MOE_ACT_SILU>());
    else if (act == MOE_ACT_GELU)
        f(std::integral_constant<int, MOE_ACT_GELU>());
    else if (act == MOE_ACT_RELU)
        f(std::integral_constant<int, MOE_ACT_RELU>());
    else
        f(std::integral_constant<int, MOE_ACT_NONE>());
}

}  // namespace dev
}  // namespace moe
