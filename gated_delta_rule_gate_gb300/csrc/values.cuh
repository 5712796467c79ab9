// values.cuh -- groups of V adjacent values, read and written as one word.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace gdn {

// V adjacent values as they are stored: one word of up to 16 bytes (fp32: V / 4 of
// them), so that they can be on their way while others are worked on.
template <typename T, int V>
struct Words {
    static constexpr int kBytes = V * (int)sizeof(T) > 16 ? 16 : V * (int)sizeof(T);
    static constexpr int kCount = V * (int)sizeof(T) / kBytes;
    using type = std::conditional_t<
        V == 1, T,
        std::conditional_t<sizeof(T) == 4, std::conditional_t<V == 2, float2, float4>,
                           std::conditional_t<V == 8, uint4, std::conditional_t<V == 4, uint2, uint32_t>>>>;
    type w[kCount];

    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < kCount; ++i) w[i] = reinterpret_cast<const type *>(p)[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kCount; ++i) w[i] = type{};
    }
    __device__ __forceinline__ void get(float (&v)[V]) const {
        if constexpr (V == 1) {
            v[0] = static_cast<float>(w[0]);
        } else if constexpr (sizeof(T) == 4 && V == 2) {
            v[0] = w[0].x, v[1] = w[0].y;
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < kCount; ++i)
                v[4 * i] = w[i].x, v[4 * i + 1] = w[i].y, v[4 * i + 2] = w[i].z, v[4 * i + 3] = w[i].w;
        } else {
            static_assert(V == 8 || V == 4 || V == 2, "16-bit groups");
            const uint32_t *u = reinterpret_cast<const uint32_t *>(&w[0]);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                uint32_t q = u[i];
                float2 f;
                if constexpr (std::is_same<T, __half>::value) f = __half22float2(*reinterpret_cast<__half2 *>(&q));
                else f = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&q));
                v[2 * i] = f.x, v[2 * i + 1] = f.y;
            }
        }
    }
};

// V values of type T at p, which is aligned to V of them (to 16 bytes from there on).
template <typename T, int V>
__device__ __forceinline__ void load_values(const T *p, float (&v)[V]) {
    Words<T, V> w;
    w.load(p);
    w.get(v);
}

template <typename T, int V>
__device__ __forceinline__ void store_values(T *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = static_cast<T>(v[0]);
    } else if constexpr (sizeof(T) == 4 && V == 2) {
        *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
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
        else if constexpr (V == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(p) = w[0];
    }
}

// V adjacent columns c, ... of a row of n values (n % V == 0); zeros from column n on.
template <typename T, int V>
struct Columns : Words<T, V> {
    __device__ __forceinline__ void load(const T *row, int c, int n) {
        this->zero();
        if (c < n) Words<T, V>::load(row + c);
    }
};
template <typename T, int V>
__device__ __forceinline__ void load_columns(const T *row, int c, int n, float (&v)[V]) {
    Columns<T, V> q;
    q.load(row, c, n);
    q.get(v);
}
template <typename T, int V>
__device__ __forceinline__ void store_columns(T *row, int c, int n, const float (&v)[V]) {
    if (c < n) store_values<T, V>(row + c, v);
}

}  // namespace gdn
