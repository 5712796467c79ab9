// adamw.cu -- gdn_adamw: one AdamW step over many tensors.
//
// One kernel a group of tensors (up to kMany of one kind, whose table travels as a kernel
// argument, so nothing is copied to the device first).  Elements are taken by rows of 256,
// a warp a row, 8 elements a lane in two groups of four, which makes every access of fp32,
// 16-bit and 8-bit values a whole word over adjacent lanes; a row is also the block of
// 8-bit states that shares its scales, so that the largest of a block is a maximum over
// one warp.  Everything is read once and written once.  Bound by HBM: 4.0e8 bf16 elements
// with fp32 copies and states (28 bytes each) 1636 us, 6.9 TB/s; with 8-bit states (10 bytes
// each) 673 us, 6.0 TB/s, where the 52 instructions of an element fill 78 % of the issue slots.
#include <math.h>
#include <string.h>

#include <cuda_fp8.h>

#include <memory>
#include <new>
#include <utility>

#include "launch.h"
#include "ptx.cuh"
#include "status.h"
#include "values.cuh"

namespace gdn {
namespace adamw {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMany = 400, kFew = 32;  // tensors of a table: one of few keeps the launch's argument small
constexpr int kStretch = 8;            // rows of a warp (16: 119 us for 113, 2^26 elements with 8-bit states)
constexpr int kRow = GDN_ADAMW_BLOCK;
constexpr int kGroups = kRow / 128;  // of four adjacent elements a lane
static_assert(kRow == 256, "a lane's two groups of four");

struct Tensor {
    void *p;
    const void *g;
    void *m, *v;
    float *ms, *vs, *master;
    int64_t n, first;  // elements; its first row, counted over the table
    uint8_t p_type, g_type, whole;  // gdn_dtypes; all its tensors begin at 16-byte addresses
};
template <int MAX>
struct Table {
    Tensor t[MAX];
    int64_t rows;
    int count, stretch, slots;  // tensors, rows of a block, slots of a warp (fewer than its ring where its rows are)
};
// What the step is made of, and the two places of which the host need not know.
struct Step {
    float beta1, rest1, beta2, rest2;  // rest = 1 - beta, rounded from 64 bits
    float log_beta1, log_beta2;
    float lr, weight_decay, eps, max_norm, norm_eps;
    float zero;       // -0
    float c1, root2;  // 1 - beta1^t and sqrt(1 - beta2^t) where step is NULL
    const int64_t *step;
    const float *lr_at;
    const float *norm;
    int32_t *err;
};
// The same for every element.  The divisor of m is taken 2^24 times as large, and the rate with it: where
// a root is 0 the divisor is eps, which may be a subnormal number, of which the fast reciprocal
// is infinite.  (Any other root is above 2^-75.)
constexpr float kUp = 0x1p24f;
struct Factors {
    float clip, rate, decay, unroot, eps;  // rate, unroot and eps kUp times as large
};

template <int MAX>
__device__ __forceinline__ int find_tensor(const Table<MAX> &tab, int64_t row) {
    int lo = 0, hi = tab.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.t[mid].first <= row) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ uint32_t raw1(const void *base, int type, int64_t at) {
    return type == GDN_DTYPE_F32 ? static_cast<const uint32_t *>(base)[at] : static_cast<const uint16_t *>(base)[at];
}
__device__ __forceinline__ float2 widen2(uint32_t w, int type) {
    return type == GDN_DTYPE_F16 ? __half22float2(*reinterpret_cast<__half2 *>(&w))
                                 : __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&w));
}
__device__ __forceinline__ float widen1(uint32_t r, int type) {
    return type == GDN_DTYPE_F32 ? __uint_as_float(r) : widen2(r, type).x;
}
__device__ __forceinline__ void put1(void *base, int type, int64_t at, float v) {
    if (type == GDN_DTYPE_F32) static_cast<float *>(base)[at] = v;
    else if (type == GDN_DTYPE_F16) static_cast<__half *>(base)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(base)[at] = __float2bfloat16_rn(v);
}
// e4m3 codes, two in a half-word, first lowest.
__device__ __forceinline__ float2 decode2(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
__device__ __forceinline__ uint32_t encode2(float2 v) { return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3); }

// Pairs of elements throughout (packed fp32).  What 8-bit codes depend on is rounded one by
// one, in the formula's order: codes and scales are then a function of the definition
// alone, and a value that lies between two codes falls where it does for anyone who
// evaluates it so.  What only p takes (root and reciprocal) is approximate, 2 ulp each, which leaves
// less than p's own rounding.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float root_of(float v) {
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// Of a number that is not subnormal.
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// a b + c d with each product and the sum rounded.  Of packed products and a sum the compiler
// makes an fma, whatever rounding they name; so each product is an fma with a -0 that it
// does not know to be one.
__device__ __forceinline__ float2 mix(float a, float2 b, float c, float2 d, float zero) {
    return __fadd2_rn(__ffma2_rn(both(a), b, both(zero)), __ffma2_rn(both(c), d, both(zero)));
}
// A root that is up to 2 ulp off, rounded: one step of Newton's method, whose residual
// v - s^2 an fma gives without error (Markstein 1990; of v below 2^-104, gradients of 1e-15, the
// residual is rounded too and the root within an ulp).  2^26 bf16 elements with 8-bit states take
// 116 us so, and 124 with __fsqrt_rn.
__device__ __forceinline__ float2 rounded_root(float2 s, float2 v) {
    const float2 r = __ffma2_rn(__fmul2_rn(both(-1.f), s), s, v);
    const float2 h = make_float2(reciprocal(fmaxf(s.x, 0x1p-80f)), reciprocal(fmaxf(s.y, 0x1p-80f)));
    return __ffma2_rn(r, __fmul2_rn(both(0.5f), h), s);
}

// A pair of elements: p, m and v (in 32 bits) and their gradients.  Returns the roots of v,
// approximate ones.
__device__ __forceinline__ float2 update(const Step &st, const Factors &f, float2 g, float2 &p, float2 &m, float2 &v) {
    g = __fmul2_rn(g, both(f.clip));
    m = mix(st.beta1, m, st.rest1, g, st.zero);
    v = mix(st.beta2, v, st.rest2, __fmul2_rn(g, g), st.zero);
    const float2 root = make_float2(root_of(v.x), root_of(v.y));
    const float2 den = __ffma2_rn(root, both(f.unroot), both(f.eps));
    const float2 q = __fmul2_rn(m, make_float2(reciprocal(den.x), reciprocal(den.y)));
    p = __ffma2_rn(both(-f.rate), q, __ffma2_rn(both(-f.decay), p, p));
    return root;
}

// A block's scale and the reciprocal with which quotients are formed.
struct Scale {
    float s, inv;
};
// The larger one, or NaN where there is one: a block with a NaN says so by its scale.
__device__ __forceinline__ float larger(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ Scale scale_of(const float2 (&y)[4]) {
    float a = 0x1p-100f;
#pragma unroll
    for (int i = 0; i < 4; ++i) a = larger(a, larger(fabsf(y[i].x), fabsf(y[i].y)));
    // numbers that are not negative compare as their bits do, and this NaN (0x7fffffff) is above them
    a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
    const float s = a * (1.f / 448.f);
    return {s, __frcp_rn(s)};
}
// y / s as a division rounds it: one product and two fma (Markstein), s.inv being rounded.
__device__ __forceinline__ float2 quotient(float2 y, const Scale &s) {
    const float2 q = __fmul2_rn(y, both(s.inv));
    return __ffma2_rn(__ffma2_rn(q, both(-s.s), y), both(s.inv), q);
}
__device__ __forceinline__ float at_least(float q, float root) { return root > 0.f ? fmaxf(q, 0x1p-9f) : q; }
__device__ __forceinline__ float2 root_code(float2 root, const Scale &s) {
    const float2 q = quotient(root, s);
    return make_float2(at_least(q.x, root.x), at_least(q.y, root.y));
}

// Four adjacent values, of a row in shared or global memory and to one in global memory.
template <typename T>
__device__ __forceinline__ void get4(const unsigned char *row, int at, float2 *v) {
    if constexpr (sizeof(T) == 4) {
        const float4 w = *reinterpret_cast<const float4 *>(row + 4 * at);
        v[0] = make_float2(w.x, w.y), v[1] = make_float2(w.z, w.w);
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(row + 2 * at);
        constexpr int type = std::is_same<T, __half>::value ? GDN_DTYPE_F16 : GDN_DTYPE_BF16;
        v[0] = widen2(w.x, type), v[1] = widen2(w.y, type);
    }
}
template <typename T>
__device__ __forceinline__ void put4(void *base, int64_t at, const float2 *v) {
    const float f[4] = {v[0].x, v[0].y, v[1].x, v[1].y};
    store_values<T, 4>(static_cast<T *>(base) + at, f);
}

// A whole row of 256 elements; a lane has elements 4 lane + 128 j ... + 3.  With 8-bit states rows
// come through shared memory (cp.async), several on their way a warp without a register:
// 2^26 bf16 elements take 174, 137, 116 us with two, three, four of them (and took half as
// much again with the next row in registers).
// P, G: the types of parameters and gradients; MASTER: there are fp32 copies.
template <bool EIGHT, typename P, bool MASTER, typename G>
struct Whole {
    using Kept = std::conditional_t<MASTER, float, P>;  // what the step is taken on
    static constexpr int kP = sizeof(Kept) * kRow, kG = sizeof(G) * kRow;
    static constexpr int kState = EIGHT ? kRow : 4 * kRow;
    static constexpr int kBytes = kP + kG + 2 * kState + 16;  // and the scales
    // as many rows a warp as leave room for four blocks an SM
    static constexpr int kSlots = 54 * 1024 / (kWarps * kBytes);
    static constexpr int kSmem = EIGHT ? kWarps * kSlots * kBytes : 0;

    template <int N>
    static __device__ __forceinline__ void copy(unsigned char *to, const void *from, int64_t row, int lane) {
        static_assert(N % 512 == 0, "16 bytes a lane");
        const char *src = static_cast<const char *>(from) + row * N;
#pragma unroll
        for (int o = 0; o < N; o += 512) ptx::cp_async16(to + o + 16 * lane, src + o + 16 * lane, 16);
    }
    static __device__ __forceinline__ void load(unsigned char *slot, const Tensor &t, int64_t row, int lane) {
        copy<kP>(slot, MASTER ? static_cast<const void *>(t.master) : t.p, row, lane);
        copy<kG>(slot + kP, t.g, row, lane);
        unsigned char *m = slot + kP + kG;
        // half a warp each
        const char *src = static_cast<const char *>(lane < 16 ? t.m : t.v) + row * kRow;
        ptx::cp_async16(m + 16 * lane, src + 16 * (lane & 15), 16);
        if (lane < 2) ptx::cp_async4(m + 2 * kState + 4 * lane, (lane ? t.vs : t.ms) + row);
    }
    static __device__ __forceinline__ void step(const unsigned char *slot, const Step &st, const Factors &f,
                                                const Tensor &t, int64_t row, int lane) {
        const unsigned char *sp, *sg, *sm, *sv;
        float2 p[4], m[4], v[4], root[4];
        float ms = 0.f, vs = 0.f;
        if constexpr (EIGHT) {
            sp = slot, sg = sp + kP, sm = sg + kG, sv = sm + kState;
            ms = *reinterpret_cast<const float *>(sv + kState);
            vs = *reinterpret_cast<const float *>(sv + kState + 4);
        } else {
            sp = static_cast<const unsigned char *>(MASTER ? static_cast<const void *>(t.master) : t.p) + row * kP;
            sg = static_cast<const unsigned char *>(t.g) + row * kG;
            sm = static_cast<const unsigned char *>(t.m) + row * kState;
            sv = static_cast<const unsigned char *>(t.v) + row * kState;
        }
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            const int e = 4 * lane + 128 * j;
            float2 g[2];
            get4<G>(sg, e, g);
            get4<Kept>(sp, e, p + 2 * j);
            if constexpr (EIGHT) {
                const uint32_t cm = *reinterpret_cast<const uint32_t *>(sm + e);
                const uint32_t cv = *reinterpret_cast<const uint32_t *>(sv + e);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    m[2 * j + h] = __fmul2_rn(decode2(cm >> 16 * h & 0xffff), both(ms));
                    v[2 * j + h] = __fmul2_rn(decode2(cv >> 16 * h & 0xffff), both(vs));
                    v[2 * j + h] = __fmul2_rn(v[2 * j + h], v[2 * j + h]);
                }
            } else {
                get4<float>(sm, e, m + 2 * j);
                get4<float>(sv, e, v + 2 * j);
            }
#pragma unroll
            for (int i = 2 * j; i < 2 * j + 2; ++i) {
                root[i] = update(st, f, g[i - 2 * j], p[i], m[i], v[i]);
                if (EIGHT) root[i] = rounded_root(root[i], v[i]);
            }
        }
        if (EIGHT) __syncwarp();  // the slot has been read
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            const int64_t e = row * kRow + 4 * lane + 128 * j;
            if (MASTER) put4<float>(t.master, e, p + 2 * j);
            put4<P>(t.p, e, p + 2 * j);
            if constexpr (!EIGHT) {
                put4<float>(t.m, e, m + 2 * j);
                put4<float>(t.v, e, v + 2 * j);
            }
        }
        if constexpr (EIGHT) {
            const Scale qm = scale_of(m), qv = scale_of(root);
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                const int64_t e = row * (kRow / 4) + lane + 32 * j;
                static_cast<uint32_t *>(t.m)[e] =
                    encode2(quotient(m[2 * j], qm)) | encode2(quotient(m[2 * j + 1], qm)) << 16;
                static_cast<uint32_t *>(t.v)[e] =
                    encode2(root_code(root[2 * j], qv)) | encode2(root_code(root[2 * j + 1], qv)) << 16;
            }
            if (lane == 0) t.ms[row] = qm.s, t.vs[row] = qv.s;
        }
    }
};

// A row of up to 256 elements at any address: a lane has elements lane + 32 i.  2^26 bf16 elements all of
// whose rows come here, because a tensor is not at a 16-byte address, take 314 us (278 in whole rows) with fp32
// copies and states, 323 (114) with 8-bit states.
template <bool EIGHT>
__device__ __forceinline__ void loose_row(const Step &st, const Factors &f, const Tensor &t, int64_t at, int lane) {
    const int n = (int)(t.n - at < kRow ? t.n - at : kRow);
    const int pt = t.master ? GDN_DTYPE_F32 : t.p_type, gt = t.g_type;
    const void *pin = t.master ? t.master : t.p;
    uint8_t *mc = static_cast<uint8_t *>(t.m), *vc = static_cast<uint8_t *>(t.v);
    uint32_t gr[8], pr[8], mr[8], vr[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t e = at + lane + 32 * i;
        gr[i] = pr[i] = mr[i] = vr[i] = 0;
        if (lane + 32 * i < n) {
            gr[i] = raw1(t.g, gt, e);
            pr[i] = raw1(pin, pt, e);
            mr[i] = EIGHT ? mc[e] : static_cast<const uint32_t *>(t.m)[e];
            vr[i] = EIGHT ? vc[e] : static_cast<const uint32_t *>(t.v)[e];
        }
    }
    float2 p[4], m[4], v[4], root[4];
    const float ms = EIGHT ? t.ms[at / kRow] : 0.f, vs = EIGHT ? t.vs[at / kRow] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 g = make_float2(widen1(gr[2 * i], gt), widen1(gr[2 * i + 1], gt));
        p[i] = make_float2(widen1(pr[2 * i], pt), widen1(pr[2 * i + 1], pt));
        if (EIGHT) {
            m[i] = __fmul2_rn(decode2(mr[2 * i] | mr[2 * i + 1] << 8), both(ms));
            v[i] = __fmul2_rn(decode2(vr[2 * i] | vr[2 * i + 1] << 8), both(vs));
            v[i] = __fmul2_rn(v[i], v[i]);
        } else {
            m[i] = make_float2(__uint_as_float(mr[2 * i]), __uint_as_float(mr[2 * i + 1]));
            v[i] = make_float2(__uint_as_float(vr[2 * i]), __uint_as_float(vr[2 * i + 1]));
        }
        root[i] = update(st, f, g, p[i], m[i], v[i]);
        if (EIGHT) root[i] = rounded_root(root[i], v[i]);
    }
    Scale sm = {0.f, 0.f}, sv = {0.f, 0.f};
    if (EIGHT) {
        // zeros beyond the end have states of zero (with an eps of 0 only their p is NaN)
        sm = scale_of(m), sv = scale_of(root);
        if (lane == 0) t.ms[at / kRow] = sm.s, t.vs[at / kRow] = sv.s;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t cm = EIGHT ? encode2(quotient(m[i], sm)) : 0, cv = EIGHT ? encode2(root_code(root[i], sv)) : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t e = at + lane + 32 * (2 * i + h);
            if (lane + 32 * (2 * i + h) >= n) continue;
            const float y = h ? p[i].y : p[i].x;
            if (t.master) t.master[e] = y;
            put1(t.p, t.p_type, e, y);
            if (EIGHT) {
                mc[e] = (uint8_t)(cm >> 8 * h), vc[e] = (uint8_t)(cv >> 8 * h);
            } else {
                static_cast<float *>(t.m)[e] = h ? m[i].y : m[i].x;
                static_cast<float *>(t.v)[e] = h ? v[i].y : v[i].x;
            }
        }
    }
}

__device__ __forceinline__ bool whole_row(const Tensor &t, int64_t row) { return t.whole && (row + 1) * kRow <= t.n; }

// A block has a stretch of adjacent rows, which its warps take in turn, and there are as
// many blocks as stretches: SMs are not equally fast (equal shares of a persistent grid took
// 235 us in place of 218 for 2^26 bf16 elements with fp32 states).
template <bool EIGHT, typename P, bool MASTER, typename G, int MAX>
__global__ void __launch_bounds__(kThreads, EIGHT ? 4 : 2) adamw_kernel(const __grid_constant__ Table<MAX> tab,
                                                                        const __grid_constant__ Step st) {
    extern __shared__ __align__(16) unsigned char slots[];
    ptx::grid_wait();
    Factors f;
    f.clip = 1.f;
    if (st.norm) {
        const float norm = *st.norm;
        if (!isfinite(norm)) {  // gradients that say nothing: the step is not taken
            if (blockIdx.x == 0 && threadIdx.x == 0 && st.err) atomicOr(st.err, kErrNonfinite);
            return;
        }
        f.clip = fminf(1.f, st.max_norm * __frcp_rn(norm + st.norm_eps));
    }
    const float lr = st.lr_at ? *st.lr_at : st.lr;
    float c1 = st.c1, root2 = st.root2;
    if (st.step) {
        const int64_t s = *st.step;
        const float k = s < 1 ? 1.f : (float)s;
        c1 = -expm1f(k * st.log_beta1);
        root2 = sqrtf(-expm1f(k * st.log_beta2));
    }
    f.rate = kUp * __fdiv_rn(lr, c1);
    f.decay = lr * st.weight_decay;
    f.unroot = __fdiv_rn(kUp, root2);
    f.eps = kUp * st.eps;
    using Rows = Whole<EIGHT, P, MASTER, G>;
    constexpr int N = EIGHT ? Rows::kSlots : 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t row = (int64_t)blockIdx.x * tab.stretch + warp;
    const int64_t stop = row - warp + tab.stretch < tab.rows ? row - warp + tab.stretch : tab.rows;
    int i = find_tensor(tab, row);
    // slots, of rows ahead of this one (8-bit states)
    unsigned char *mine = slots + warp * tab.slots * Rows::kBytes;
    int64_t ahead = row;
    int ia = i, at = 0, to = 0;
    auto request = [&] {
        while (ia + 1 < tab.count && tab.t[ia + 1].first <= ahead) ++ia;
        const Tensor &t = tab.t[ia];
        if (ahead < stop && whole_row(t, ahead - t.first))
            Rows::load(mine + to * Rows::kBytes, t, ahead - t.first, lane);
        ptx::cp_async_commit();
        ahead += kWarps;
        to = to + 1 == N ? 0 : to + 1;
    };
    if constexpr (EIGHT) {
        const Tensor t = tab.t[i];
        if (row < stop && whole_row(t, stop - 1 - t.first)) {
            // a stretch of one tensor's whole rows, its addresses kept (looked up for each row: 140 us for 116)
            const int rows = (int)((stop - row + kWarps - 1) / kWarps);
            const int64_t r0 = row - t.first;
#pragma unroll 1
            for (int k = 0; k < N - 1; ++k) {
                if (k < rows) Rows::load(mine + k * Rows::kBytes, t, r0 + k * kWarps, lane);
                ptx::cp_async_commit();
            }
            to = N - 1;
#pragma unroll 1
            for (int k = 0; k < rows; ++k) {
                if (k + N - 1 < rows) Rows::load(mine + to * Rows::kBytes, t, r0 + (k + N - 1) * kWarps, lane);
                ptx::cp_async_commit();
                ptx::cp_async_wait<N - 1>();
                __syncwarp();
                Rows::step(mine + at * Rows::kBytes, st, f, t, r0 + k * kWarps, lane);
                at = at + 1 == N ? 0 : at + 1;
                to = to + 1 == N ? 0 : to + 1;
            }
            return;
        }
#pragma unroll 1
        for (int k = 0; k < N - 1; ++k) request();
    }
    for (; row < stop; row += kWarps) {
        if constexpr (EIGHT) {
            request();
            ptx::cp_async_wait<N - 1>();
            __syncwarp();
        }
        while (i + 1 < tab.count && tab.t[i + 1].first <= row) ++i;
        const Tensor &t = tab.t[i];
        if (whole_row(t, row - t.first)) Rows::step(mine + at * Rows::kBytes, st, f, t, row - t.first, lane);
        else loose_row<EIGHT>(st, f, t, (row - t.first) * kRow, lane);
        at = at + 1 == N ? 0 : at + 1;
    }
}

// Tensors of one kind share a kernel: the types of parameters and of gradients, and
// whether there is a copy.  (An fp32 parameter with a copy goes element by element.)
constexpr int kKinds = 15;
int kind_of(const gdn_adamw_args *a, int i) {
    const int p = a->param_dtypes[i], copied = p != GDN_DTYPE_F32 && a->master && a->master[i];
    return (p + 2 * copied) * 3 + a->grad_dtypes[i];
}
static_assert(GDN_DTYPE_F32 == 0 && GDN_DTYPE_F16 == 1 && GDN_DTYPE_BF16 == 2, "kinds count types");
template <int TYPE>
using TypeOf = std::conditional_t<TYPE == GDN_DTYPE_F32, float, std::conditional_t<TYPE == GDN_DTYPE_F16, __half, __nv_bfloat16>>;

// Fills a table with tensors of a kind from i on; returns the first that was not looked at.
template <int MAX>
int fill(const gdn_adamw_args *a, int i, int kind, Table<MAX> *tab) {
    tab->count = 0, tab->rows = 0;
    for (; i < a->count && tab->count < MAX; ++i) {
        if (a->sizes[i] == 0 || kind_of(a, i) != kind) continue;
        Tensor &t = tab->t[tab->count++];
        t.p = a->params[i], t.g = a->grads[i], t.m = a->exp_avg[i], t.v = a->exp_avg_sq[i];
        const bool eight = a->state_dtype == GDN_DTYPE_E4M3;
        t.ms = eight ? a->exp_avg_scales[i] : nullptr;
        t.vs = eight ? a->exp_avg_sq_scales[i] : nullptr;
        t.master = a->master ? a->master[i] : nullptr;
        t.n = a->sizes[i];
        t.first = tab->rows;
        t.p_type = (uint8_t)a->param_dtypes[i], t.g_type = (uint8_t)a->grad_dtypes[i];
        t.whole = aligned(t.p, 16) && aligned(t.g, 16) && aligned(t.m, 16) && aligned(t.v, 16) &&
                  aligned(t.master, 16) && !(t.master && t.p_type == GDN_DTYPE_F32);
        tab->rows += (t.n + kRow - 1) / kRow;
    }
    // rows of a warp: so few that they reach all SMs (six blocks each), up to kStretch
    const int64_t warps = (int64_t)kWarps * sm_count() * 6;
    int64_t each = (tab->rows + warps - 1) / warps;
    each = each < 1 ? 1 : each > kStretch ? kStretch : each;
    while (tab->rows / (each * kWarps) >= 1LL << 31) each *= 2;
    tab->stretch = (int)each * kWarps;
    return i;
}

template <int KIND, bool EIGHT, int MAX>
cudaError_t launch(Table<MAX> &tab, const Step &st, cudaStream_t stream) {
    constexpr int p = KIND / 3;
    constexpr bool copied = p > 2;
    using P = TypeOf<(copied ? p - 2 : p)>;
    using G = TypeOf<KIND % 3>;
    using Rows = Whole<EIGHT, P, copied, G>;
    const auto kernel = adamw_kernel<EIGHT, P, copied, G, MAX>;
    const cudaError_t e = smem_attr((const void *)kernel, Rows::kSmem);
    if (e != cudaSuccess) return e;
    const int each = tab.stretch / kWarps;
    tab.slots = each < Rows::kSlots ? each : Rows::kSlots;
    const size_t smem = EIGHT ? kWarps * tab.slots * Rows::kBytes : 0;
    const int64_t blocks = (tab.rows + tab.stretch - 1) / tab.stretch;
    return launch_early(kernel, (unsigned)blocks, kThreads, smem, stream, tab, st);
}

template <bool EIGHT, int MAX, int... KINDS>
cudaError_t run(const gdn_adamw_args *a, const Step &st, cudaStream_t stream, std::integer_sequence<int, KINDS...>) {
    cudaError_t (*const launchers[])(Table<MAX> &, const Step &, cudaStream_t) = {launch<KINDS, EIGHT, MAX>...};
    bool present[kKinds] = {};
    for (int i = 0; i < a->count; ++i)
        if (a->sizes[i] > 0) present[kind_of(a, i)] = true;
    Table<MAX> tab;
    for (int kind = 0; kind < kKinds; ++kind) {
        for (int i = 0; present[kind] && i < a->count;) {
            i = fill<MAX>(a, i, kind, &tab);
            if (tab.rows == 0) continue;
            const cudaError_t e = launchers[kind](tab, st, stream);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}
template <bool EIGHT>
cudaError_t run(const gdn_adamw_args *a, const Step &st, cudaStream_t stream) {
    const auto kinds = std::make_integer_sequence<int, kKinds>();
    return a->count <= kFew ? run<EIGHT, kFew>(a, st, stream, kinds) : run<EIGHT, kMany>(a, st, stream, kinds);
}

}  // namespace adamw
}  // namespace gdn

namespace {

using gdn::aligned;
using gdn::fail;

bool finite_from(double v, double least) { return isfinite(v) && v >= least; }

// No two tensors that a step writes begin at one address: one that is listed twice (tied weights, a state
// for all) would be stepped by two warps at once.  By a table of the addresses, which costs the
// host 10 ns a weight; sorting them, to see parts of tensors too, took 50 to 120.
gdn_status check_apart(const gdn_adamw_args *a) {
    const struct {
        const char *name;
        const void *const *at;
    } lists[] = {{"params", (const void *const *)a->params},
                 {"exp_avg", (const void *const *)a->exp_avg},
                 {"exp_avg_sq", (const void *const *)a->exp_avg_sq},
                 {"exp_avg_scales", (const void *const *)a->exp_avg_scales},
                 {"exp_avg_sq_scales", (const void *const *)a->exp_avg_sq_scales},
                 {"master", (const void *const *)a->master}};
    int64_t most = 0;
    for (const auto &l : lists) most += l.at ? a->count : 0;
    int bits = 6;
    while ((1LL << bits) < most + most / 2) ++bits;  // places, a third of them empty at least
    constexpr int kSome = 9;
    uintptr_t some[1 << kSome], *seen = some;
    std::unique_ptr<uintptr_t[]> more;
    if (bits > kSome) {
        more.reset(new (std::nothrow) uintptr_t[(size_t)1 << bits]);
        seen = more.get();
        if (!seen) return fail(GDN_ERR_CUDA, "no host memory for %d tensors", a->count);
    }
    memset(seen, 0, sizeof(uintptr_t) << bits);
    for (const auto &l : lists) {
        if (!l.at) continue;
        for (int i = 0; i < a->count; ++i) {
            const uintptr_t at = reinterpret_cast<uintptr_t>(l.at[i]);
            if (!at || a->sizes[i] == 0) continue;
            // an fp32 weight may be its own copy: both are given the same value by the same thread
            if (l.at == (const void *const *)a->master && l.at[i] == a->params[i] &&
                a->param_dtypes[i] == GDN_DTYPE_F32)
                continue;
            uint64_t place = (uint64_t)at * 0x9e3779b97f4a7c15u >> (64 - bits);
            while (seen[place] && seen[place] != at) place = (place + 1) & ((1ull << bits) - 1);
            if (seen[place]) {
                for (const auto &o : lists)
                    for (int k = 0; o.at && k < a->count; ++k)
                        if (a->sizes[k] > 0 && o.at[k] == l.at[i])
                            return fail(GDN_ERR_INVALID, "%s[%d] is %s[%d]: one tensor twice", l.name, i, o.name, k);
            }
            seen[place] = at;
        }
    }
    return GDN_OK;
}

gdn_status validate(const gdn_adamw_args *a) {
    if (!a) return fail(GDN_ERR_INVALID, "args is NULL");
    if (a->count < 0) return fail(GDN_ERR_INVALID, "count must be >= 0");
    if (a->state_dtype != GDN_DTYPE_F32 && a->state_dtype != GDN_DTYPE_E4M3)
        return fail(GDN_ERR_INVALID, "state_dtype must be F32 or E4M3");
    if (!a->step_device && a->step < 1) return fail(GDN_ERR_INVALID, "step must be >= 1 (the first step is 1)");
    if (!a->lr_device && !finite_from(a->lr, 0)) return fail(GDN_ERR_INVALID, "lr must be >= 0 and finite");
    if (!(a->beta1 >= 0 && a->beta1 < 1) || !(a->beta2 >= 0 && a->beta2 < 1))
        return fail(GDN_ERR_INVALID, "beta1 and beta2 must be in [0, 1)");
    if (!finite_from(a->eps, 0)) return fail(GDN_ERR_INVALID, "eps must be >= 0 and finite");
    if (!finite_from(a->weight_decay, 0)) return fail(GDN_ERR_INVALID, "weight_decay must be >= 0 and finite");
    if (a->grad_norm && !finite_from(a->max_norm, 0)) return fail(GDN_ERR_INVALID, "max_norm must be >= 0 and finite");
    if (a->grad_norm && !finite_from(a->norm_eps, 0)) return fail(GDN_ERR_INVALID, "norm_eps must be >= 0 and finite");
    const bool eight = a->state_dtype == GDN_DTYPE_E4M3;
    if (a->count > 0 && (!a->params || !a->grads || !a->exp_avg || !a->exp_avg_sq || !a->sizes || !a->param_dtypes ||
                         !a->grad_dtypes))
        return fail(GDN_ERR_INVALID, "params, grads, exp_avg, exp_avg_sq, sizes and dtypes are required");
    if (a->count > 0 && eight != (a->exp_avg_scales != nullptr && a->exp_avg_sq_scales != nullptr))
        return fail(GDN_ERR_INVALID, eight ? "8-bit states need exp_avg_scales and exp_avg_sq_scales"
                                           : "scales given without 8-bit states");
    if (!eight && (a->exp_avg_scales || a->exp_avg_sq_scales))
        return fail(GDN_ERR_INVALID, "scales given without 8-bit states");
    const size_t es = eight ? 1 : 4;
    for (int i = 0; i < a->count; ++i) {
        const int pt = a->param_dtypes[i], gt = a->grad_dtypes[i];
        if ((pt != GDN_DTYPE_F32 && pt != GDN_DTYPE_F16 && pt != GDN_DTYPE_BF16) ||
            (gt != GDN_DTYPE_F32 && gt != GDN_DTYPE_F16 && gt != GDN_DTYPE_BF16))
            return fail(GDN_ERR_INVALID, "tensor %d: unknown dtype %d, %d", i, pt, gt);
        if (a->sizes[i] < 0) return fail(GDN_ERR_INVALID, "tensor %d: size must be >= 0", i);
        if (a->sizes[i] > (1LL << 40)) return fail(GDN_ERR_UNSUPPORTED, "tensor %d: more than 2^40 elements", i);
        if (a->sizes[i] == 0) continue;
        if (!a->params[i] || !a->grads[i] || !a->exp_avg[i] || !a->exp_avg_sq[i] ||
            (eight && (!a->exp_avg_scales[i] || !a->exp_avg_sq_scales[i])))
            return fail(GDN_ERR_INVALID, "tensor %d: NULL", i);
        if (!aligned(a->params[i], pt == GDN_DTYPE_F32 ? 4 : 2) || !aligned(a->grads[i], gt == GDN_DTYPE_F32 ? 4 : 2) ||
            !aligned(a->exp_avg[i], es) || !aligned(a->exp_avg_sq[i], es) ||
            (eight && (!aligned(a->exp_avg_scales[i], 4) || !aligned(a->exp_avg_sq_scales[i], 4))) ||
            (a->master && !aligned(a->master[i], 4)))
            return fail(GDN_ERR_INVALID, "tensor %d is not aligned to its element size", i);
    }
    if (!aligned(a->step_device, 8) || !aligned(a->lr_device, 4) || !aligned(a->grad_norm, 4) ||
        !aligned(a->error_word, 4))
        return fail(GDN_ERR_INVALID, "a pointer is not aligned to its element size");
    return check_apart(a);
}

}  // namespace

extern "C" gdn_status gdn_adamw(const gdn_adamw_args *a, gdn_stream stream) {
    const gdn_status st = validate(a);
    if (st != GDN_OK) return st;
    gdn::adamw::Step s = {};
    s.beta1 = (float)a->beta1, s.rest1 = (float)(1 - a->beta1);
    s.beta2 = (float)a->beta2, s.rest2 = (float)(1 - a->beta2);
    s.lr = (float)a->lr, s.weight_decay = (float)a->weight_decay, s.eps = (float)a->eps;
    if (a->eps > 0) s.eps = fmaxf(s.eps, 0x1p-149f);  // an eps stays one
    s.zero = -0.f;
    s.max_norm = (float)a->max_norm, s.norm_eps = (float)a->norm_eps;
    // beta = 0 has logarithm -inf, and 1 - beta^t = 1
    s.log_beta1 = (float)log(a->beta1), s.log_beta2 = (float)log(a->beta2);
    if (!a->step_device) {
        s.c1 = (float)-expm1((double)a->step * log(a->beta1));
        s.root2 = (float)sqrt(-expm1((double)a->step * log(a->beta2)));
    }
    s.step = a->step_device, s.lr_at = a->lr_device, s.norm = a->grad_norm, s.err = a->error_word;
    cudaStream_t q = (cudaStream_t)stream;
    return gdn::cuda_status(a->state_dtype == GDN_DTYPE_E4M3 ? gdn::adamw::run<true>(a, s, q)
                                                             : gdn::adamw::run<false>(a, s, q));
}
