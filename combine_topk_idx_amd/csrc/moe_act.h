// Activations of the bf16 expert layer and their slopes, on the device.
#pragma once

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

__device__ __forceinline__ float act_value(int act, float v)
{
    if (act == MOE_ACT_SILU)
        return v / (1.0f + expf(-v));
    if (act == MOE_ACT_GELU)
        return v / (1.0f + expf(-gelu_z(near(v))));
    if (act == MOE_ACT_RELU)
        return v < 0.0f ? 0.0f : v;
    return v;
}

// The value f and the slope d of an activation at v.
__device__ __forceinline__ void act_both(int act, float v, float &f, float &d)
{
    if (act == MOE_ACT_SILU) {
        const float s = 1.0f / (1.0f + expf(-v));
        f = v * s;
        d = s + f * (1.0f - s);
    } else if (act == MOE_ACT_GELU) {
        const float c = near(v);
        const float s = 1.0f / (1.0f + expf(-gelu_z(c)));
        f = v * s;
        d = s + c * s * (1.0f - s) * (kGeluLinear + 3.0f * kGeluCubic * c * c);
    } else if (act == MOE_ACT_RELU) {
        f = v < 0.0f ? 0.0f : v;
        d = v <= 0.0f ? 0.0f : v > 0.0f ? 1.0f : v;
    } else {
        f = v;
        d = 1.0f;
    }
}

}  // namespace dev
}  // namespace moe
