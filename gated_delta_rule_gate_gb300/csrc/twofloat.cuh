// twofloat.cuh -- numbers of about 48 bits as unevaluated sums of two fp32 values
// (Dekker's and Knuth's error-free sums and products), for the few places where fp32
// is not enough: the device's fp64 rate is so low that one block's fp64 sum of 1,000
// values, with its root, took 5 us.
#pragma once

#include <cuda_runtime.h>

namespace gdn {

struct TwoFloat {
    float hi, lo;
};
// a + b exactly.
__device__ __forceinline__ TwoFloat two_sum(float a, float b) {
    const float s = a + b, v = s - a;
    return {s, (a - (s - v)) + (b - v)};
}
// a b exactly.
__device__ __forceinline__ TwoFloat two_product(float a, float b) {
    const float p = __fmul_rn(a, b);
    return {p, fmaf(a, b, -p)};
}
__device__ __forceinline__ TwoFloat normalised(float hi, float lo) {
    const float s = hi + lo;
    return {s, lo - (s - hi)};
}
__device__ __forceinline__ TwoFloat operator+(TwoFloat a, TwoFloat b) {
    const TwoFloat s = two_sum(a.hi, b.hi);
    return normalised(s.hi, s.lo + (a.lo + b.lo));
}
__device__ __forceinline__ TwoFloat operator-(TwoFloat a) { return {-a.hi, -a.lo}; }
__device__ __forceinline__ TwoFloat operator*(TwoFloat a, TwoFloat b) {
    const TwoFloat p = two_product(a.hi, b.hi);
    return normalised(p.hi, fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, p.lo)));
}
__device__ __forceinline__ TwoFloat operator/(TwoFloat a, float b) {
    const float q = a.hi / b;
    return normalised(q, (fmaf(-q, b, a.hi) + a.lo) / b);
}
__device__ __forceinline__ TwoFloat warp_sum(TwoFloat v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const TwoFloat w = {__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)};
        v = v + w;
    }
    return v;
}

}  // namespace gdn
