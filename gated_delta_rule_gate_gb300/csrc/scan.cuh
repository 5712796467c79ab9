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
    int wide;              // the inputs' rows begin on 16-byte addresses
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

// ---------------------------------------------------------------- arithmetic
// Two channels at a time.  The gates' functions are the larger part of the
// kernels' instructions, so they are written for packed fp32 and few special
// function units; their relative errors stay within a few 2^-24 where the state
// remembers (a near 1), since a state of M tokens' memory carries M times a's.
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 operator+(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 operator*(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

__device__ __forceinline__ float ex2(float v) {  // 2^v
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float root(float v) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// sigmoid(z) = 1 / (1 + e^-z).
__device__ __forceinline__ float2 sigmoid(float2 z) {
    const float2 d = make_float2(ex2(-kLog2e * z.x), ex2(-kLog2e * z.y)) + splat(1.f);
    return make_float2(reciprocal(d.x), reciprocal(d.y));
}

// softplus(z) = max(z, 0) + log1p(u), u = e^-|z| in (0, 1].  log1p(u) / u is a
// polynomial of degree 8 fitted on [0, 1] (weighted least squares at Chebyshev
// nodes, toward the least largest relative error): 1.7e-7 with fp32 rounding.
__device__ __forceinline__ float2 softplus(float2 z, float2 &u) {
    u = make_float2(ex2(-kLog2e * fabsf(z.x)), ex2(-kLog2e * fabsf(z.y)));
    float2 r = splat(0.00523266801610589f);
    r = fma2(r, u, splat(-0.029505133628845215f));
    r = fma2(r, u, splat(0.07822578400373459f));
    r = fma2(r, u, splat(-0.1366323083639145f));
    r = fma2(r, u, splat(0.19106000661849976f));
    r = fma2(r, u, splat(-0.2484298050403595f));
    r = fma2(r, u, splat(0.3331909775733948f));
    r = fma2(r, u, splat(-0.4999949336051941f));
    r = fma2(r, u, splat(0.9999999403953552f));
    return fma2(r, u, make_float2(fmaxf(z.x, 0.f), fmaxf(z.y, 0.f)));
}

// e^g - 1: for |g| <= 1/2 a polynomial times g (degree 6, fitted as above, 1.2e-7),
// else 2^(g log2 e) - 1.  1 + it is then e^g without a bias where g is near 0.
__device__ __forceinline__ float2 exp_minus_1(float2 g) {
    float2 r = splat(0.00019841187167912722f);
    r = fma2(r, g, splat(0.0013997324276715517f));
    r = fma2(r, g, splat(0.008333634585142136f));
    r = fma2(r, g, splat(0.041665319353342056f));
    r = fma2(r, g, splat(0.16666662693023682f));
    r = fma2(r, g, splat(0.5000000596046448f));
    r = fma2(r, g, splat(1.f)) * g;
    const float2 t = g * splat(kLog2e);
    const float2 e = make_float2(ex2(t.x), ex2(t.y)) + splat(-1.f);
    return make_float2(fabsf(g.x) <= 0.5f ? r.x : e.x, fabsf(g.y) <= 0.5f ? r.y : e.y);
}

// What a token's gates come to: a = exp(g), the input's scale n, and m = a - 1.
template <bool RAW>
__device__ __forceinline__ float2 log_decay(float2 z, float2 bias, float2 scale) {
    float2 u;
    return RAW ? scale * softplus(z + bias, u) : z;
}
// n^2 = 1 - a^2 = -m (2 + m) with m = a - 1, and 0 where a > 1.
__device__ __forceinline__ float2 unit_scale(float2 m) {
    const float2 q = m * (splat(-2.f) + make_float2(-m.x, -m.y));
    return make_float2(root(fmaxf(q.x, 0.f)), root(fmaxf(q.y, 0.f)));
}
// a and u = n i x of a token.
template <bool RAW, bool BETA, int MODE>
__device__ __forceinline__ void token_map(float2 x, float2 z, float2 y, float2 bias, float2 scale, bool sig, float2 &a,
                                          float2 &u) {
    const float2 m = exp_minus_1(log_decay<RAW>(z, bias, scale));
    a = m + splat(1.f);
    u = x;
    if constexpr (BETA) u = u * (sig ? sigmoid(y) : y);
    if constexpr (MODE == kLerp) u = u * make_float2(-m.x, -m.y);
    if constexpr (MODE == kUnit) u = u * unit_scale(m);
}

// What the gradient needs of one token's gates: a, n, dn/dg, i, di/dbeta,
// softplus, dg/ddecay.
struct Terms {
    float2 a, n, dn, i, di, soft, dgdz;
};
template <bool RAW, bool BETA, int MODE>
__device__ __forceinline__ Terms gate_terms(float2 z, float2 y, float2 bias, float2 scale, bool sig) {
    Terms t;
    float2 g = z;
    t.soft = splat(0.f);
    t.dgdz = splat(1.f);
    if constexpr (RAW) {
        float2 u;
        z = z + bias;
        t.soft = softplus(z, u);
        g = scale * t.soft;
        // sigmoid(z) = 1 / (1 + u) for z >= 0, u / (1 + u) below
        const float2 d = u + splat(1.f), r = make_float2(reciprocal(d.x), reciprocal(d.y)), l = u * r;
        t.dgdz = scale * make_float2(z.x >= 0.f ? r.x : l.x, z.y >= 0.f ? r.y : l.y);
    }
    const float2 m = exp_minus_1(g);
    t.a = m + splat(1.f);
    t.n = splat(1.f);
    t.dn = splat(0.f);
    if constexpr (MODE == kLerp) {
        t.n = make_float2(-m.x, -m.y);
        t.dn = make_float2(-t.a.x, -t.a.y);
    }
    if constexpr (MODE == kUnit) {  // where n is 0 (a >= 1) its slope is taken as 0
        t.n = unit_scale(m);
        const float2 q = t.a * t.a;
        t.dn = make_float2(t.n.x > 0.f ? -q.x * reciprocal(t.n.x) : 0.f, t.n.y > 0.f ? -q.y * reciprocal(t.n.y) : 0.f);
    }
    t.i = splat(1.f);
    t.di = splat(0.f);
    if constexpr (BETA) {
        t.i = sig ? sigmoid(y) : y;
        t.di = sig ? t.i * (splat(1.f) + make_float2(-t.i.x, -t.i.y)) : splat(1.f);
    }
    return t;
}

}  // namespace scan
}  // namespace gdn
