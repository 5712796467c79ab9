// glu_math.cuh -- the activations of the gated feed-forward and their derivatives, fp32.
//
// exp and the quotients are the fast ones (a few 2^-23 of the value): results are
// rounded to 16 bits.  Each form keeps its relative precision where the function or
// its derivative is small.
#pragma once

#include <cuda_runtime.h>

#include "../../include/gdn.h"

namespace gdn {
namespace glu {

constexpr float kRootHalf = 0.70710678118654752f;    // sqrt(1 / 2)
constexpr float kPhi0 = 0.39894228040143268f;        // 1 / sqrt(2 pi)
constexpr float kTanhScale = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// act(g).  0.5 (1 + tanh z) is sigmoid(2 z), and 0.5 (1 + erf(g / sqrt 2)) is
// 0.5 erfc(-g / sqrt 2), which lose nothing to cancellation for negative g.
__device__ __forceinline__ float activation(float g, int act) {
    switch (act) {
        case GDN_ACT_SILU: return g * sigmoid(g);
        case GDN_ACT_GELU: return 0.5f * g * erfcf(-g * kRootHalf);
        case GDN_ACT_GELU_TANH: return g * sigmoid(kTanhScale * fmaf(kTanhCube * g * g, g, g));
        case GDN_ACT_RELU: return g < 0.f ? 0.f : g;  // NaN stays
        default: return sigmoid(g);
    }
}

// act(g) and act'(g).
__device__ __forceinline__ float2 activation_slope(float g, int act) {
    if (act == GDN_ACT_RELU) return make_float2(g < 0.f ? 0.f : g, g > 0.f ? 1.f : g <= 0.f ? 0.f : g);
    if (act == GDN_ACT_GELU) {
        const float cdf = 0.5f * erfcf(-g * kRootHalf);
        return make_float2(g * cdf, fmaf(g, kPhi0 * __expf(-0.5f * g * g), cdf));
    }
    // the rest by s = sigmoid(z) and r = 1 - s, each from the same e^-|z| <= 1
    const float z = act == GDN_ACT_GELU_TANH ? kTanhScale * fmaf(kTanhCube * g * g, g, g) : g;
    const float e = __expf(-fabsf(z)), big = __fdividef(1.f, 1.f + e), small = e * big;
    const float s = z >= 0.f ? big : small, r = z >= 0.f ? small : big;
    if (act == GDN_ACT_SIGMOID) return make_float2(s, s * r);
    if (act == GDN_ACT_SILU) return make_float2(g * s, s * fmaf(g, r, 1.f));
    // z' = kTanhScale (1 + 3 kTanhCube g^2); beyond |g| = 30 s r is 0 and z' may be infinite
    const float c = fminf(fmaxf(g, -30.f), 30.f);
    return make_float2(g * s, fmaf(c * s * r, kTanhScale * fmaf(3.f * kTanhCube * c, c, 1.f), s));
}

}  // namespace glu
}  // namespace gdn
