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

// What the block needs of a gate g: act(g), and its derivative where SLOPE.
struct FfnGate {
    float act, slope;
};
template <bool SLOPE>
__device__ __forceinline__ FfnGate ffn_gate(int act, float g) {
    FfnGate r{0.f, 0.f};
    if (act == CE_ACT_GELU) {
        const float phi = 0.5f * erfcf(-0.70710678f * g);
        r.act = g * phi;
        if (SLOPE) r.slope = phi + g * 0.39894228f * ex2(-0.5f * kLog2e * g * g);
    } else {
        const bool silu = act == CE_ACT_SILU;
        const float q = ffn_logistic(silu ? g : kGelu2k * g * (1.f + kGeluC * g * g));
        r.act = g * q;
        if (SLOPE) {
            const float d = q * (1.f - q);  // 0 where g g may overflow
            r.slope = q + (d > 0.f ? g * d * (silu ? 1.f : kGelu2k * (1.f + 3.f * kGeluC * g * g)) : 0.f);
        }
    }
    return r;
}

}  // namespace gbce
