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
    int wide;              // every tensor's rows begin on 16-byte addresses
    int groups, per;       // groups of requests that a cluster takes side by side, requests in one
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
// Channels c, c + 1 at p (the second where ok1), one by one.
template <typename T>
__device__ __forceinline__ pair_t<T> load_pair(const T *p, bool ok1) {
    pair_t<T> v;
    T *e = reinterpret_cast<T *>(&v);
    e[0] = *p;
    e[1] = p[ok1 ? 1 : 0];  // unused where there is none
    return v;
}
// A warp writes the first n of a row's 64 channels at p, a lane two of them, whatever
// the row's alignment: of a 16-bit row that begins between two words a lane writes its
// second channel and its neighbour's first as one.
template <typename T>
__device__ __forceinline__ void store_row(T *p, float2 v, int lane, int n) {
    if constexpr (sizeof(T) == 4) {
        if (2 * lane < n) p[2 * lane] = v.x;
        if (2 * lane + 1 < n) p[2 * lane + 1] = v.y;
    } else {
        const uint32_t mine = pack<T>(v);
        uint16_t *e = reinterpret_cast<uint16_t *>(p);
        if (!(reinterpret_cast<uintptr_t>(p) & 2u)) {
            if (2 * lane + 1 < n) reinterpret_cast<uint32_t *>(p)[lane] = mine;
            else if (2 * lane < n) e[2 * lane] = (uint16_t)mine;
        } else {
            const uint32_t w = __funnelshift_r(mine, __shfl_down_sync(0xffffffffu, mine, 1), 16);
            if (lane < 31 && 2 * lane + 2 < n) *reinterpret_cast<uint32_t *>(e + 2 * lane + 1) = w;
            else if (2 * lane + 1 < n) e[2 * lane + 1] = (uint16_t)w;
            if (lane == 0 && n > 0) e[0] = (uint16_t)mine;
        }
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
// owned by a request and in [lo, hi), first and last of it; lane k holds the state
// row of token t + k.  `seen` is the last request met, so that a tile inside it takes
// no search.
struct Tokens {
    unsigned own, first, last;
    int row;
};
struct Seen {
    int t0 = 0, t1 = 0, row = -1;
};
__device__ __forceinline__ Tokens look_up(const Args &p, int lo, int hi, int t, int n, int lane, Seen &seen) {
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
    if (lane < n && tk >= lo && tk < hi) {
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
// remembers (a near 1), since a state of M tokens' memory carries M times a's, and
// grow with |g| (see exponential) where it forgets.
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

__device__ __forceinline__ float2 operator-(float2 a) { return a * splat(-1.f); }

// sigmoid(z) = 1 / (1 + e^-z).
__device__ __forceinline__ float2 sigmoid(float2 z) {
    const float2 t = z * splat(-kLog2e);
    const float2 d = make_float2(ex2(t.x), ex2(t.y)) + splat(1.f);
    return make_float2(reciprocal(d.x), reciprocal(d.y));
}

// softplus(z) = max(z, 0) + log1p(u), u = e^-|z| in (0, 1].  log1p(u) / u is a
// polynomial of degree 8 fitted on [0, 1] (weighted least squares at Chebyshev
// nodes, toward the least largest relative error): 1.7e-7 with fp32 rounding.
__device__ __forceinline__ float2 softplus(float2 z) {
    const float2 u = make_float2(ex2(-kLog2e * fabsf(z.x)), ex2(-kLog2e * fabsf(z.y)));
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

// e^g, and m = e^g - 1 without cancellation: for |g| <= 1/5 a polynomial times g (degree 4,
// fitted as above, 1.4e-7) and 1 + it, which has no bias where g is near 0; else 2^(g log2 e),
// whose error is (4 + 1.25 |g|) 2^-24 of itself (ex2.approx, the product's rounding), and that
// less 1.  Below 2^-126 it is 0.  1 + m for all g would leave a small decay on steps of 2^-24.
struct Exp {
    float2 a, m;
};
__device__ __forceinline__ Exp exponential(float2 g) {
    float2 r = splat(0.008333331905305386f);
    r = fma2(r, g, splat(0.04173609986901283f));
    r = fma2(r, g, splat(0.16666696965694427f));
    r = fma2(r, g, splat(0.4999993145465851f));
    r = fma2(r, g, splat(1.f)) * g;
    const float2 t = g * splat(kLog2e), e = make_float2(ex2(t.x), ex2(t.y));
    const float2 a = r + splat(1.f), m = e + splat(-1.f);
    const bool x = fabsf(g.x) <= 0.2f, y = fabsf(g.y) <= 0.2f;
    return {make_float2(x ? a.x : e.x, y ? a.y : e.y), make_float2(x ? r.x : m.x, y ? r.y : m.y)};
}

template <bool RAW>
__device__ __forceinline__ float2 log_decay(float2 z, float2 bias, float2 scale) {
    return RAW ? scale * softplus(z + bias) : z;
}
// n^2 = 1 - a^2 = -m (2 + m) with m = a - 1, and 0 where a > 1.
__device__ __forceinline__ float2 unit_scale(float2 m) {
    const float2 q = m * fma2(m, splat(-1.f), splat(-2.f));
    return make_float2(root(fmaxf(q.x, 0.f)), root(fmaxf(q.y, 0.f)));
}

// What a token's gates come to: g, a = exp(g), the input's scale n, its gate i, and in
// the raw arm softplus(z).
struct Gates {
    float2 g, a, n, i, soft;
};
template <bool RAW, bool BETA, int MODE>
__device__ __forceinline__ Gates token_gates(float2 z, float2 y, float2 bias, float2 scale, bool sig) {
    Gates t;
    t.soft = RAW ? softplus(z + bias) : splat(0.f);
    t.g = RAW ? scale * t.soft : z;
    const Exp e = exponential(t.g);
    t.a = e.a;
    t.n = MODE == kLerp ? -e.m : (MODE == kUnit ? unit_scale(e.m) : splat(1.f));
    t.i = BETA ? (sig ? sigmoid(y) : y) : splat(1.f);
    return t;
}
// n i x.
template <bool BETA, int MODE>
__device__ __forceinline__ float2 scaled(float2 x, float2 n, float2 i) {
    if (BETA) x = x * i;
    return MODE == kNone ? x : x * n;
}

}  // namespace scan
}  // namespace gdn
