// The activations of the gated feed-forward block and their derivatives, in
// fp32: silu(g) = g s(g), gelu(g) = g Phi(g) (the normal distribution
// function), gelu_tanh(g) = g s(2 k (g + c g^3)), k = sqrt(2 / pi), c =
// 0.044715, which is 0.5 g (1 + tanh(...)); s the logistic function.
#pragma once

#include <cstdint>

#include "ce_device.cuh"
#include "gbce.h"

namespace gbce {

__device__ __forceinline__ float ffn_logistic(float z) {
    return __fdividef(1.f, 1.f + ex2(-z * kLog2e));
}

constexpr float kGelu2k = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;

__device__ __forceinline__ float ffn_act(int act, float g) {
    if (act == CE_ACT_SILU) return g * ffn_logistic(g);
    if (act == CE_ACT_GELU) return g * (0.5f * erfcf(-0.70710678f * g));
    return g * ffn_logistic(kGelu2k * g * (1.f + kGeluC * g * g));
}

// d act / d g
__device__ __forceinline__ float ffn_slope(int act, float g) {
    if (act == CE_ACT_SILU) {
        const float q = ffn_logistic(g);
        return q * (1.f + g * (1.f - q));
    }
    if (act == CE_ACT_GELU)
        return 0.5f * erfcf(-0.70710678f * g) + g * 0.39894228f * ex2(-0.5f * kLog2e * g * g);
    const float q = ffn_logistic(kGelu2k * g * (1.f + kGeluC * g * g));
    return q + g * q * (1.f - q) * kGelu2k * (1.f + 3.f * kGeluC * g * g);
}

}  // namespace gbce
