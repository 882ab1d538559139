// product_device.cuh -- device-side helpers of the products and the
// feed-forward block.
#pragma once

#include "layer_device.cuh"
#include "product_internal.h"

namespace hyena {

// act(g) of the gated block (HYENA_ACT_*), and with it act'(g).
template <int kAct>
__device__ __forceinline__ float activation(float g)
{
    if constexpr (kAct == HYENA_ACT_SILU) {
        return g / (1.f + expf(-g));
    } else if constexpr (kAct == HYENA_ACT_GELU) {
        return 0.5f * g * (1.f + erff(g * 0.70710678118654752f));
    } else if constexpr (kAct == HYENA_ACT_GELU_TANH) {
        return 0.5f * g * (1.f + tanhf(0.79788456080286536f * fmaf(0.044715f * g * g, g, g)));
    } else {
        return g;
    }
}

template <int kAct>
__device__ __forceinline__ float2 activation_slope(float g)
{
    if constexpr (kAct == HYENA_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-g));
        return make_float2(g * s, s * fmaf(g, 1.f - s, 1.f));
    } else if constexpr (kAct == HYENA_ACT_GELU) {
        const float c = 0.5f * (1.f + erff(g * 0.70710678118654752f));
        return make_float2(g * c, fmaf(g, 0.39894228040143268f * expf(-0.5f * g * g), c));
    } else if constexpr (kAct == HYENA_ACT_GELU_TANH) {
        const float t = tanhf(0.79788456080286536f * fmaf(0.044715f * g * g, g, g));
        const float in = 0.79788456080286536f * fmaf(3.f * 0.044715f * g, g, 1.f);
        return make_float2(0.5f * g * (1.f + t), 0.5f * (1.f + t) + 0.5f * g * (1.f - t * t) * in);
    } else {
        return make_float2(g, 1.f);
    }
}

__device__ __forceinline__ uint16_t bf16_bits(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

}  // namespace hyena
