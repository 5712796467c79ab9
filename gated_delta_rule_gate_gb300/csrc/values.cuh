// values.cuh -- groups of V adjacent values, read and written as one word.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace gdn {

// V values of type T at p (V > 1: 16 bytes, or 32 as two, aligned to 16).
template <typename T, int V>
__device__ __forceinline__ void load_values(const T *p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = static_cast<float>(*p);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 r = *reinterpret_cast<const float4 *>(p + i);
            v[i] = r.x, v[i + 1] = r.y, v[i + 2] = r.z, v[i + 3] = r.w;
        }
    } else {
        static_assert(V == 8 || V == 4, "16-bit groups");
        uint32_t w[V / 2];
        if constexpr (V == 8) {
            const uint4 r = *reinterpret_cast<const uint4 *>(p);
            w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
        } else {
            const uint2 r = *reinterpret_cast<const uint2 *>(p);
            w[0] = r.x, w[1] = r.y;
        }
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            float2 f;
            if constexpr (std::is_same<T, __half>::value) f = __half22float2(*reinterpret_cast<__half2 *>(&w[i]));
            else f = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&w[i]));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_values(T *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = static_cast<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (std::is_same<T, __half>::value) {
                __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<uint32_t *>(&h);
            } else {
                __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<uint32_t *>(&h);
            }
        }
        if constexpr (V == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

}  // namespace gdn
