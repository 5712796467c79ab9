// scan.cuh -- what the kernels of the gated linear recurrence share: the
// problem, pairs of channels, requests and state rows, the gates' arithmetic.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

namespace gdn {
namespace scan {

enum : int { kNone = 0, kLerp = 1, kUnit = 2 };  // gdn_input_scale
constexpr int kChunk = 64;                       // GDN_SCAN_CHUNK

// A validated call of gdn_scan or gdn_scan_step (and the forward half of the
// gradient's), passed by value to the kernels.
struct Args {
    int B, T, L, D, rows;  // L: tokens of a request's row in the uniform forms, 0 with cu
    int mode, sigmoid;
    int vec;               // pairs of channels can be read and written as one word
    int64_t xs, gs, bs, os;
    const void *x, *decay, *beta;
    void *o;
    const float *bias, *scale;
    const int32_t *cu, *seqlens, *slots;
    const float *init;
    float *fin, *chunk;
    int32_t *err;
};

// A validated call of gdn_scan_backward.
struct GradArgs {
    Args f;  // the forward call; chunk is read
    int64_t dos, dxs, dgs, dbs;
    const void *d_o;
    const float *dfin;
    void *dx, *dg, *db;
    float *dbias, *dscale, *dinit;
};

// Two adjacent channels of one token, as stored.
template <typename T>
struct Pair;
template <>
struct Pair<float> {
    using type = float2;
};
template <>
struct Pair<__half> {
    using type = uint32_t;
};
template <>
struct Pair<__nv_bfloat16> {
    using type = uint32_t;
};
template <typename T>
using pair_t = typename Pair<T>::type;

template <typename T>
__device__ __forceinline__ float2 unpack(pair_t<T> v) {
    if constexpr (sizeof(T) == 4) {
        return v;
    } else if constexpr (std::is_same<T, __half>::value) {
        return __half22float2(*reinterpret_cast<__half2 *>(&v));
    } else {
        return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&v));
    }
}
template <typename T>
__device__ __forceinline__ pair_t<T> pack(float2 v) {
    if constexpr (sizeof(T) == 4) {
        return v;
    } else if constexpr (std::is_same<T, __half>::value) {
        __half2 h = __floats2half2_rn(v.x, v.y);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}
template <typename T>
__device__ __forceinline__ pair_t<T> zero_pair() {
    return pack<T>(make_float2(0.f, 0.f));
}
// Channels c, c + 1 at p: one word where `vec`, else element by element, the
// second only where ok1 (the caller checks the first).
template <typename T>
__device__ __forceinline__ pair_t<T> load_pair(const T *p, bool vec, bool ok1) {
    if (vec) return __ldg(reinterpret_cast<const pair_t<T> *>(p));
    float2 v;
    v.x = static_cast<float>(p[0]);
    v.y = ok1 ? static_cast<float>(p[1]) : 0.f;
    return pack<T>(v);  // exact: the values come from T
}
template <typename T>
__device__ __forceinline__ void store_pair(T *p, float2 v, bool vec, bool ok1) {
    if (vec) {
        *reinterpret_cast<pair_t<T> *>(p) = pack<T>(v);
    } else {
        p[0] = static_cast<T>(v.x);
        if (ok1) p[1] = static_cast<T>(v.y);
    }
}
// The same for fp32 state rows, whose alignment follows the channel count alone.
__device__ __forceinline__ float2 load_state(const float *p, int c, int D) {
    return make_float2(c < D ? p[c] : 0.f, c + 1 < D ? p[c + 1] : 0.f);
}
__device__ __forceinline__ void store_state(float *p, int c, int D, float2 v) {
    if (c < D) p[c] = v.x;
    if (c + 1 < D) p[c + 1] = v.y;
}

// ---------------------------------------------------------------- requests
__device__ __forceinline__ int clamped_offset(const Args &p, int i) {
    const int v = p.cu[i];
    return v < 0 ? 0 : (v > p.T ? p.T : v);
}
// Tokens [t0, t1) of request b (see gdn_scan_args; a decreasing pair is empty).
__device__ __forceinline__ void request_tokens(const Args &p, int b, int &t0, int &t1) {
    if (p.cu) {
        t0 = clamped_offset(p, b);
        t1 = clamped_offset(p, b + 1);
        t1 = t1 < t0 ? t0 : t1;
    } else {
        t0 = b * p.L;
        int n = p.L;
        if (p.seqlens) {
            n = p.seqlens[b];
            n = n < 0 ? 0 : (n > p.L ? p.L : n);
        }
        t1 = t0 + n;
    }
}
// State row of request b, or -1 for a slot id out of range.
__device__ __forceinline__ int request_row(const Args &p, int b) {
    const int r = p.slots ? p.slots[b] : b;
    return r < 0 || r >= p.rows ? -1 : r;
}
// The request that owns token t (0 <= t < T), its tokens and state row; false
// for a token of no request.  With offsets: the last one that is <= t, so that
// of equal offsets the request that is not empty is taken.
__device__ __forceinline__ bool find_request(const Args &p, int t, int &t0, int &t1, int &row) {
    int b;
    if (p.cu) {
        int lo = 0, hi = p.B;  // cu[lo] <= t < cu[hi], as far as the search knows
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (clamped_offset(p, mid) <= t) lo = mid; else hi = mid;
        }
        b = lo;
    } else {
        b = t / p.L;
    }
    request_tokens(p, b, t0, t1);
    row = request_row(p, b);
    return t >= t0 && t < t1 && row >= 0;
}

// The tokens of a warp's tile [t, t + n), n <= 32, as masks of their places:
// owned by a request, first and last of it; lane k holds the state row of token
// t + k.  `in0`, `in1` carry the last request seen, so that a tile inside it
// takes no search.
struct Tokens {
    unsigned own, first, last;
    int row;
};
struct Seen {
    int t0 = 0, t1 = 0, row = -1;
};
__device__ __forceinline__ Tokens look_up(const Args &p, int t, int n, int lane, Seen &seen) {
    Tokens k;
    if (t > seen.t0 && t + n < seen.t1 && t >= 0) {
        k.own = seen.row >= 0 ? (n == 32 ? ~0u : (1u << n) - 1u) : 0u;
        k.first = k.last = 0u;
        k.row = seen.row;
        return k;
    }
    bool own = false, first = false, last = false;
    int t0 = 0, t1 = 0, row = -1;
    const int tk = t + lane;
    if (lane < n && tk >= 0 && tk < p.T) {
        own = find_request(p, tk, t0, t1, row);
        first = own && tk == t0;
        last = own && tk + 1 == t1;
    }
    k.own = __ballot_sync(0xffffffffu, own);
    k.first = __ballot_sync(0xffffffffu, first);
    k.last = __ballot_sync(0xffffffffu, last);
    k.row = row;
    // every lane keeps the request of the tile's last owned token
    const int src = k.own ? 31 - __clz(k.own) : 0;
    seen.t0 = __shfl_sync(0xffffffffu, t0, src);
    seen.t1 = __shfl_sync(0xffffffffu, t1, src);
    seen.row = __shfl_sync(0xffffffffu, row, src);
    if (!k.own) seen.t1 = 0;
    return k;
}

// ---------------------------------------------------------------- gates
// softplus(z) = max(z, 0) + log1p(e^-|z|).
__device__ __forceinline__ float softplus(float z) { return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))); }
__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

template <bool RAW>
__device__ __forceinline__ float log_decay(float z, float bias, float scale) {
    return RAW ? scale * softplus(z + bias) : z;
}
// What the gradient needs of one token's gates: a, n, dn/dg, i, di/dbeta,
// softplus, dg/ddecay.
struct Terms {
    float a, n, dn, i, di, soft, dgdz;
};
template <bool RAW, bool BETA, int MODE>
__device__ __forceinline__ Terms gate_terms(float z, float y, float bias, float scale, bool sig) {
    Terms t;
    float g = z;
    t.soft = 0.f;
    t.dgdz = 1.f;
    if constexpr (RAW) {
        z += bias;
        t.soft = softplus(z);
        g = scale * t.soft;
        t.dgdz = scale * sigmoid(z);
    }
    t.a = expf(g);
    t.n = 1.f;
    t.dn = 0.f;
    if constexpr (MODE == kLerp) {
        t.n = -expm1f(g);
        t.dn = -t.a;
    }
    if constexpr (MODE == kUnit) {  // where n is 0 (a >= 1) its slope is taken as 0
        t.n = sqrtf(fmaxf(0.f, -expm1f(2.f * g)));
        t.dn = t.n > 0.f ? -t.a * t.a / t.n : 0.f;
    }
    t.i = 1.f;
    t.di = 0.f;
    if constexpr (BETA) {
        t.i = sig ? sigmoid(y) : y;
        t.di = sig ? t.i * (1.f - t.i) : 1.f;
    }
    return t;
}

// n of the input x; a = exp(g).
template <int MODE>
__device__ __forceinline__ float input_scale(float g, float a) {
    if constexpr (MODE == kLerp) return -expm1f(g);
    if constexpr (MODE == kUnit) return sqrtf(fmaxf(0.f, -expm1f(2.f * g)));
    return 1.f;
}

}  // namespace scan
}  // namespace gdn
