// Activations of the gated feed-forward block: act(g) = g s(t(g)) with the
// logistic function s, t(g) = g (SiLU) or 2 sqrt(2/pi)(g + 0.044715 g^3) (the
// tanh form of GELU, since (1 + tanh z) / 2 = s(2 z)).
#pragma once

#include "common.cuh"
#include "moe_ffn_block.h"

namespace moe {

// s(t): the divide is within a few ulp of fp32, and its limits are right: for
// exp(-t) above 2^126 the quotient is 0.
__device__ __forceinline__ float logistic(float t) { return __fdividef(1.0f, 1.0f + __expf(-t)); }

constexpr float kGelu0 = 1.5957691216057308f;              // 2 sqrt(2 / pi)
constexpr float kGelu1 = 1.5957691216057308f * 0.044715f;

// t(g).  Its square stops at 10^4: s(t) is 0 or 1 long before, and t and t'
// stay finite for every finite g.
__device__ __forceinline__ float act_square(float g) { return fminf(g * g, 1.0e4f); }

// act(g) u.  g of minus infinity (s = 0) gives 0 times it, a NaN, as the formula has it.
__device__ __forceinline__ float glu(float g, float u, int act) {
    const float t = act == MOE_ACT_SILU ? g : g * (kGelu0 + kGelu1 * act_square(g));
    return g * logistic(t) * u;
}

// act(g) and act'(g) = s + act(g) (1 - s) t'(g).
__device__ __forceinline__ void act_slope(float g, int act, float& a, float& slope) {
    const float g2 = act_square(g);
    const float t = act == MOE_ACT_SILU ? g : g * (kGelu0 + kGelu1 * g2);
    const float dt = act == MOE_ACT_SILU ? 1.0f : kGelu0 + 3.0f * kGelu1 * g2;
    const float s = logistic(t);
    a = g * s;
    slope = s + a * (1.0f - s) * dt;
}

}  // namespace moe
