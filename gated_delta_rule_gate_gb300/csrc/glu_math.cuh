// glu_math.cuh -- the activations of the gated feed-forward and their derivatives, fp32.
//
// exp and the quotients are the fast ones, since results are rounded to 16 bits: an exponential
// of z is within (2 + 1.2 |z|) 2^-23 of its value, and what is formed of it within (8 + |z|) 2^-22, of GELU, whose
// z is g^2 / 2, within (8 + g^2) 2^-22.  Each form keeps that where the function or its derivative is small.
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "../../include/gdn.h"

namespace gdn {
namespace glu {

constexpr float kRootHalf = 0.70710678118654752f;    // sqrt(1 / 2)
constexpr float kPhi0 = 0.39894228040143268f;        // 1 / sqrt(2 pi)
constexpr float kTanhScale = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;
constexpr float kHalfLog2E = 0.72134752044448170f;   // log2(e) / 2

// 1 / (1 + e^-x) as 2^-24 / (2^-24 + h^2) with h = 2^-12 e^(-x / 2), within 2^-20 of the value for |x| up to
// 4, 2^-18 down to -87 (the rounding of the exponent), and two steps of 2^-149 below.  The factors are
// there for x below -87, where 1 + e^-x is above 2^126, of which the fast reciprocal is 0, or no number.
__device__ __forceinline__ float sigmoid(float x) {
    float h, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(fmaf(x, -kHalfLog2E, -12.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(h, h, 0x1p-24f)));
    return r * 0x1p-24f;
}

// Calls f with the activation as a constant: chosen once for many values.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F f) {
    switch (act) {
        case GDN_ACT_SILU: return f(std::integral_constant<int, GDN_ACT_SILU>());
        case GDN_ACT_GELU: return f(std::integral_constant<int, GDN_ACT_GELU>());
        case GDN_ACT_GELU_TANH: return f(std::integral_constant<int, GDN_ACT_GELU_TANH>());
        case GDN_ACT_RELU: return f(std::integral_constant<int, GDN_ACT_RELU>());
        default: return f(std::integral_constant<int, GDN_ACT_SIGMOID>());
    }
}

// 0.5 erfc(a) and e^(-a^2) of a >= 0, the first as t P(t) e^(-a^2) with t = 1 / (1 + 0.45 a).  P was
// fitted to 0.5 e^(a^2) erfc(a) / t for a up to 13, weighted least squares at Chebyshev nodes of t: t P(t) is within
// 7e-7 of the value when evaluated in fp32, to which e^(-a^2) adds its own error, and a^2 2^-24 for the rounding of a^2.  (With erfcf a tile of 256 x 128 results took 4.9 us more than with relu, with this 2.)
__device__ __forceinline__ float2 half_erfc(float a) {
    const float t = __fdividef(1.f, fmaf(0.45f, a, 1.f)), e = __expf(-a * a);
    float q = fmaf(0.034312523901462555f, t, -0.12385771423578262f);
    q = fmaf(q, t, 0.11093893647193909f);
    q = fmaf(q, t, 0.014052337035536766f);
    q = fmaf(q, t, 0.09759295731782913f);
    q = fmaf(q, t, 0.11303777992725372f);
    q = fmaf(q, t, 0.12697935104370117f);
    q = fmaf(q, t, 0.12694400548934937f);
    return make_float2(q * t * e, e);
}

// act(g).  0.5 (1 + tanh z) is sigmoid(2 z), and 0.5 (1 + erf(g / sqrt 2)) is
// 0.5 erfc(-g / sqrt 2) or 1 less that of the other sign, which lose nothing to cancellation for negative g.
template <int ACT>
__device__ __forceinline__ float activation(float g) {
    if constexpr (ACT == GDN_ACT_SILU) return g * sigmoid(g);
    else if constexpr (ACT == GDN_ACT_GELU) {
        const float tail = half_erfc(fabsf(g) * kRootHalf).x;
        return g * (g < 0.f ? tail : 1.f - tail);
    }
    else if constexpr (ACT == GDN_ACT_GELU_TANH) return g * sigmoid(kTanhScale * fmaf(kTanhCube * g * g, g, g));
    else if constexpr (ACT == GDN_ACT_RELU) return g < 0.f ? 0.f : g;  // NaN stays
    else return sigmoid(g);
}

// act(g) and act'(g).
template <int ACT>
__device__ __forceinline__ float2 activation_slope(float g) {
    if constexpr (ACT == GDN_ACT_RELU) {
        return make_float2(g < 0.f ? 0.f : g, g > 0.f ? 1.f : g <= 0.f ? 0.f : g);
    } else if constexpr (ACT == GDN_ACT_GELU) {
        const float2 tail = half_erfc(fabsf(g) * kRootHalf);
        const float cdf = g < 0.f ? tail.x : 1.f - tail.x;
        return make_float2(g * cdf, fmaf(g, kPhi0 * tail.y, cdf));
    } else {
        // s = sigmoid(z) and r = 1 - s, each from the same e^-|z| <= 1
        const float z = ACT == GDN_ACT_GELU_TANH ? kTanhScale * fmaf(kTanhCube * g * g, g, g) : g;
        const float e = __expf(-fabsf(z)), big = __fdividef(1.f, 1.f + e), small = e * big;
        const float s = z >= 0.f ? big : small, r = z >= 0.f ? small : big;
        if constexpr (ACT == GDN_ACT_SIGMOID) return make_float2(s, s * r);
        if constexpr (ACT == GDN_ACT_SILU) return make_float2(g * s, s * fmaf(g, r, 1.f));
        // z' = kTanhScale (1 + 3 kTanhCube g^2); beyond |g| = 30 s r is 0 and z' may be infinite
        const float c = fminf(fmaxf(g, -30.f), 30.f);
        return make_float2(g * s, fmaf(c * s * r, kTanhScale * fmaf(3.f * kTanhCube * c, c, 1.f), s));
    }
}

}  // namespace glu
}  // namespace gdn
