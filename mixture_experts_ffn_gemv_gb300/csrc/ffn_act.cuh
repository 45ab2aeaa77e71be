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

// t(g).  Its square stops at 10^4: s(t) is 0 or 1 long before.  t' stays finite
// for every finite g; t for |g| up to 4.7e35, past which it is an infinity of
// g's sign, with s(t) 1 or 0 as before.
__device__ __forceinline__ float act_square(float g) { return fminf(g * g, 1.0e4f); }

// t(g) and t'(g) of an activation known at compile time.
template <int ACT>
__device__ __forceinline__ float act_arg(float g) {
    return ACT == MOE_ACT_SILU ? g : g * (kGelu0 + kGelu1 * act_square(g));
}

// act(g) u.  g of minus infinity (s = 0) gives 0 times it, a NaN, as the formula has it.
template <int ACT>
__device__ __forceinline__ float glu(float g, float u) {
    return g * logistic(act_arg<ACT>(g)) * u;
}
__device__ __forceinline__ float glu(float g, float u, int act) {
    return act == MOE_ACT_SILU ? glu<MOE_ACT_SILU>(g, u) : glu<MOE_ACT_GELU_TANH>(g, u);
}

// act(g) and act'(g) = s + act(g) (1 - s) t'(g).
template <int ACT>
__device__ __forceinline__ void act_slope(float g, float& a, float& slope) {
    const float s = logistic(act_arg<ACT>(g));
    const float dt = ACT == MOE_ACT_SILU ? 1.0f : kGelu0 + 3.0f * kGelu1 * act_square(g);
    a = g * s;
    slope = s + a * (1.0f - s) * dt;
}
__device__ __forceinline__ void act_slope(float g, int act, float& a, float& slope) {
    if (act == MOE_ACT_SILU) act_slope<MOE_ACT_SILU>(g, a, slope);
    else act_slope<MOE_ACT_GELU_TANH>(g, a, slope);
}

// 32 elements of fp32 bits: h = act(g) u over g; or act(g) over g, u act'(g)
// over u and h as bf16 pairs.  The activation is chosen once, not per element.
template <int ACT>
__device__ __forceinline__ void glu32(uint32_t (&g)[32], const uint32_t (&u)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) g[i] = __float_as_uint(glu<ACT>(__uint_as_float(g[i]), __uint_as_float(u[i])));
}
__device__ __forceinline__ void glu32(uint32_t (&g)[32], const uint32_t (&u)[32], int act) {
    if (act == MOE_ACT_SILU) glu32<MOE_ACT_SILU>(g, u);
    else glu32<MOE_ACT_GELU_TANH>(g, u);
}
template <int ACT>
__device__ __forceinline__ void glu32_save(uint32_t (&g)[32], uint32_t (&u)[32], uint32_t (&h)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float a[2], d[2], v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float uk = __uint_as_float(u[2 * i + k]);
            float slope;
            act_slope<ACT>(__uint_as_float(g[2 * i + k]), a[k], slope);
            d[k] = uk * slope;
            v[k] = a[k] * uk;
            g[2 * i + k] = __float_as_uint(a[k]);
            u[2 * i + k] = __float_as_uint(d[k]);
        }
        h[i] = pack_bf16x2(v[0], v[1]);
    }
}
__device__ __forceinline__ void glu32_save(uint32_t (&g)[32], uint32_t (&u)[32], uint32_t (&h)[16], int act) {
    if (act == MOE_ACT_SILU) glu32_save<MOE_ACT_SILU>(g, u, h);
    else glu32_save<MOE_ACT_GELU_TANH>(g, u, h);
}

}  // namespace moe
