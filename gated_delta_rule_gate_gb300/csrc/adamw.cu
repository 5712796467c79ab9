// adamw.cu -- gdn_adamw: one AdamW step over many tensors.
//
// One kernel a group of tensors (up to kMany, whose table travels as a kernel argument,
// so nothing is copied to the device first).  Elements are taken by rows of 256, a warp
// a row, 8 elements a lane in two groups of four, which makes every access of fp32,
// 16-bit and 8-bit values a whole word over adjacent lanes; a row is also the block of
// 8-bit states that shares its scales, so that the largest of a block is a maximum over
// one warp.  Everything is read once and written once.  Bound by HBM.
#include <math.h>

#include <cuda_fp8.h>

#include "launch.h"
#include "ptx.cuh"
#include "status.h"
#include "values.cuh"

namespace gdn {
namespace adamw {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlocks = 152 * 8;
constexpr int kMany = 440, kFew = 32;
constexpr int kRow = GDN_ADAMW_BLOCK;
constexpr int kGroups = kRow / 128;  // of four adjacent elements a lane
static_assert(kRow == 256, "a lane's two groups of four");
// Rows that a block takes at a time.
constexpr int kChunk = 4 * kWarps, kSmallChunk = kWarps;
constexpr int64_t kSmall = 1 << 22;

struct Tensor {
    void *p;
    const void *g;
    void *m, *v;
    float *ms, *vs, *master;
    int64_t n;
    int32_t first;  // its first chunk, counted over the table
    uint8_t p_type, g_type, whole;  // gdn_dtypes; groups of four are words in all its tensors
};
template <int MAX>
struct Table {
    Tensor t[MAX];
    int count, chunks, chunk;  // tensors, chunks, rows of a chunk
};
// What the step is made of, and the two places of which the host need not know.
struct Step {
    float beta1, rest1, beta2, rest2;  // rest = 1 - beta, rounded from 64 bits
    float log_beta1, log_beta2;
    float lr, weight_decay, eps, max_norm, norm_eps;
    float c1, root2;  // 1 - beta1^t and sqrt(1 - beta2^t) where step is NULL
    const int64_t *step;
    const float *lr_at;
    const float *norm;
    int32_t *err;
};
// The same for every element.
struct Factors {
    float clip, rate, decay, unroot, eps;
};

template <int MAX>
__device__ __forceinline__ int find_tensor(const Table<MAX> &tab, int chunk) {
    int lo = 0, hi = tab.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.t[mid].first <= chunk) lo = mid; else hi = mid;
    }
    return lo;
}

// Four values as they are stored (16-bit ones in the first half).
__device__ __forceinline__ uint4 raw4(const void *base, int type, int64_t at) {
    if (type == GDN_DTYPE_F32) return *reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + at);
    const uint2 h = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + at);
    return make_uint4(h.x, h.y, 0, 0);
}
__device__ __forceinline__ uint32_t raw1(const void *base, int type, int64_t at) {
    return type == GDN_DTYPE_F32 ? static_cast<const uint32_t *>(base)[at] : static_cast<const uint16_t *>(base)[at];
}
__device__ __forceinline__ void widen2(uint32_t w, int type, float *v) {
    const float2 f = type == GDN_DTYPE_F16 ? __half22float2(*reinterpret_cast<__half2 *>(&w))
                                           : __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&w));
    v[0] = f.x, v[1] = f.y;
}
__device__ __forceinline__ void widen4(const uint4 &r, int type, float *v) {
    if (type == GDN_DTYPE_F32) {
        v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
    } else {
        widen2(r.x, type, v);
        widen2(r.y, type, v + 2);
    }
}
__device__ __forceinline__ float widen1(uint32_t r, int type) {
    if (type == GDN_DTYPE_F32) return __uint_as_float(r);
    float v[2];
    widen2(r, type, v);
    return v[0];
}
__device__ __forceinline__ void put4(void *base, int type, int64_t at, const float (&v)[4]) {
    if (type == GDN_DTYPE_F32) store_values<float, 4>(static_cast<float *>(base) + at, v);
    else if (type == GDN_DTYPE_F16) store_values<__half, 4>(static_cast<__half *>(base) + at, v);
    else store_values<__nv_bfloat16, 4>(static_cast<__nv_bfloat16 *>(base) + at, v);
}
__device__ __forceinline__ void put1(void *base, int type, int64_t at, float v) {
    if (type == GDN_DTYPE_F32) static_cast<float *>(base)[at] = v;
    else if (type == GDN_DTYPE_F16) static_cast<__half *>(base)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(base)[at] = __float2bfloat16_rn(v);
}
// e4m3 codes, four in a word, first lowest.
__device__ __forceinline__ void decode4(uint32_t w, float *v) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ uint32_t encode4(const float *v) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// A block's scale and the reciprocal with which quotients are formed.
struct Scale {
    float s, inv;
};
__device__ __forceinline__ Scale scale_of(const float (&y)[8]) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(y[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const float s = __fdiv_rn(fmaxf(a, 0x1p-100f), 448.f);
    return {s, __frcp_rn(s)};
}
// y / s as a division rounds it: one product and two fma.
__device__ __forceinline__ float quotient(float y, const Scale &s) {
    const float q = y * s.inv;
    return fmaf(fmaf(-q, s.s, y), s.inv, q);
}

// One element: p, m and v (in 32 bits) and its gradient.
__device__ __forceinline__ void update(const Step &st, const Factors &f, float g, float &p, float &m, float &v,
                                       float &root) {
    g *= f.clip;
    m = fmaf(st.beta1, m, st.rest1 * g);
    v = fmaf(st.beta2, v, st.rest2 * g * g);
    root = sqrtf(v);
    p = fmaf(-f.decay, p, p) - f.rate * (m / fmaf(root, f.unroot, f.eps));
}

// A row of up to 256 elements from `at` on.
template <bool EIGHT, bool WHOLE>
__device__ __forceinline__ void row_step(const Step &st, const Factors &f, const Tensor &t, int64_t at) {
    const int lane = threadIdx.x & 31;
    const int n = (int)(t.n - at < kRow ? t.n - at : kRow);
    const int pt = t.master ? GDN_DTYPE_F32 : t.p_type, gt = t.g_type;
    const void *pin = t.master ? t.master : t.p;
    const uint8_t *mc = static_cast<const uint8_t *>(t.m), *vc = static_cast<const uint8_t *>(t.v);
    float g[8], p[8], m[8], v[8], root[8];
    float ms = 0.f, vs = 0.f;
    if (EIGHT) ms = t.ms[at / kRow], vs = t.vs[at / kRow];
    // WHOLE: elements 4 lane + 128 j ...; else lane + 32 i, zeros beyond the end
    if (WHOLE) {
        uint4 gr[kGroups], pr[kGroups], mr[kGroups], vr[kGroups];
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            const int64_t e = at + 4 * lane + 128 * j;
            gr[j] = raw4(t.g, gt, e);
            pr[j] = raw4(pin, pt, e);
            if (EIGHT) {
                mr[j].x = *reinterpret_cast<const uint32_t *>(mc + e);
                vr[j].x = *reinterpret_cast<const uint32_t *>(vc + e);
            } else {
                mr[j] = raw4(t.m, GDN_DTYPE_F32, e);
                vr[j] = raw4(t.v, GDN_DTYPE_F32, e);
            }
        }
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            widen4(gr[j], gt, g + 4 * j);
            widen4(pr[j], pt, p + 4 * j);
            if (EIGHT) {
                decode4(mr[j].x, m + 4 * j);
                decode4(vr[j].x, v + 4 * j);
            } else {
                widen4(mr[j], GDN_DTYPE_F32, m + 4 * j);
                widen4(vr[j], GDN_DTYPE_F32, v + 4 * j);
            }
        }
    } else {
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
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[i] = widen1(gr[i], gt);
            p[i] = widen1(pr[i], pt);
            if (EIGHT) {
                float q[4];
                decode4(mr[i] | vr[i] << 8, q);
                m[i] = q[0], v[i] = q[1];
            } else {
                m[i] = __uint_as_float(mr[i]), v[i] = __uint_as_float(vr[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (EIGHT) {
            m[i] *= ms;
            v[i] *= vs;
            v[i] *= v[i];
        }
        update(st, f, g[i], p[i], m[i], v[i], root[i]);
        // beyond the end nothing has a say in the scales (with eps 0 it may be NaN)
        if (EIGHT && !WHOLE && lane + 32 * i >= n) m[i] = root[i] = 0.f;
    }
    if (EIGHT) {
        const Scale sm = scale_of(m), sv = scale_of(root);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[i] = quotient(m[i], sm);
            v[i] = root[i] > 0.f ? fmaxf(quotient(root[i], sv), 0x1p-9f) : root[i];
        }
        if (lane == 0) t.ms[at / kRow] = sm.s, t.vs[at / kRow] = sv.s;
    }
    if (WHOLE) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            const int64_t e = at + 4 * lane + 128 * j;
            const float(&pj)[4] = *reinterpret_cast<const float(*)[4]>(p + 4 * j);
            if (t.master) store_values<float, 4>(t.master + e, pj);
            put4(t.p, t.p_type, e, pj);
            if (EIGHT) {
                *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(t.m) + e) = encode4(m + 4 * j);
                *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(t.v) + e) = encode4(v + 4 * j);
            } else {
                store_values<float, 4>(static_cast<float *>(t.m) + e, *reinterpret_cast<const float(*)[4]>(m + 4 * j));
                store_values<float, 4>(static_cast<float *>(t.v) + e, *reinterpret_cast<const float(*)[4]>(v + 4 * j));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t e = at + lane + 32 * i;
            if (lane + 32 * i >= n) continue;
            if (t.master) t.master[e] = p[i];
            put1(t.p, t.p_type, e, p[i]);
            if (EIGHT) {
                const float q[4] = {m[i], v[i], 0.f, 0.f};
                const uint32_t c = encode4(q);
                static_cast<uint8_t *>(t.m)[e] = (uint8_t)c;
                static_cast<uint8_t *>(t.v)[e] = (uint8_t)(c >> 8);
            } else {
                static_cast<float *>(t.m)[e] = m[i];
                static_cast<float *>(t.v)[e] = v[i];
            }
        }
    }
}

template <bool EIGHT, int MAX>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<MAX> tab,
                                                         const __grid_constant__ Step st) {
    ptx::grid_wait();
    Factors f;
    f.clip = 1.f;
    if (st.norm) {
        const float norm = *st.norm;
        if (!isfinite(norm)) {  // gradients that say nothing: the step is not taken
            if (blockIdx.x == 0 && threadIdx.x == 0 && st.err) atomicOr(st.err, kErrNonfinite);
            return;
        }
        f.clip = fminf(1.f, __fdiv_rn(st.max_norm, norm + st.norm_eps));
    }
    const float lr = st.lr_at ? *st.lr_at : st.lr;
    float c1 = st.c1, root2 = st.root2;
    if (st.step) {
        const int64_t s = *st.step;
        const float k = s < 1 ? 1.f : (float)s;
        c1 = -expm1f(k * st.log_beta1);
        root2 = sqrtf(-expm1f(k * st.log_beta2));
    }
    f.rate = __fdiv_rn(lr, c1);
    f.decay = lr * st.weight_decay;
    f.unroot = __fdiv_rn(1.f, root2);
    f.eps = st.eps;
    const int warp = threadIdx.x >> 5;
    for (int chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
        const Tensor &t = tab.t[find_tensor(tab, chunk)];
        const int64_t row = (int64_t)(chunk - t.first) * tab.chunk;
        for (int r = warp; r < tab.chunk; r += kWarps) {
            const int64_t at = (row + r) * kRow;
            if (at >= t.n) break;
            if (t.whole && at + kRow <= t.n) row_step<EIGHT, true>(st, f, t, at);
            else row_step<EIGHT, false>(st, f, t, at);
        }
    }
}

bool words(const void *p, int type) { return aligned(p, type == GDN_DTYPE_F32 ? 16 : type == GDN_DTYPE_E4M3 ? 4 : 8); }

// Fills a table with tensors i, i + 1, ...; returns the first that is not in it.
template <int MAX>
int fill(const gdn_adamw_args *a, int i, int chunk, Table<MAX> *tab) {
    tab->count = tab->chunks = 0;
    tab->chunk = chunk;
    for (; i < a->count && tab->count < MAX; ++i) {
        if (a->sizes[i] == 0) continue;
        const int64_t per = (int64_t)chunk * kRow, chunks = (a->sizes[i] + per - 1) / per;
        if (tab->chunks + chunks > (1LL << 30)) break;
        Tensor &t = tab->t[tab->count++];
        t.p = a->params[i], t.g = a->grads[i], t.m = a->exp_avg[i], t.v = a->exp_avg_sq[i];
        const bool eight = a->state_dtype == GDN_DTYPE_E4M3;
        t.ms = eight ? a->exp_avg_scales[i] : nullptr;
        t.vs = eight ? a->exp_avg_sq_scales[i] : nullptr;
        t.master = a->master ? a->master[i] : nullptr;
        t.n = a->sizes[i];
        t.first = tab->chunks;
        t.p_type = (uint8_t)a->param_dtypes[i], t.g_type = (uint8_t)a->grad_dtypes[i];
        t.whole = words(t.p, t.p_type) && words(t.g, t.g_type) && words(t.m, a->state_dtype) &&
                  words(t.v, a->state_dtype) && words(t.master, GDN_DTYPE_F32);
        tab->chunks += (int)chunks;
    }
    return i;
}

template <bool EIGHT, int MAX>
cudaError_t run(const gdn_adamw_args *a, const Step &st, cudaStream_t stream) {
    int64_t elements = 0;
    for (int j = 0; j < a->count; ++j) elements += a->sizes[j];
    const int chunk = elements <= kSmall ? kSmallChunk : kChunk;
    Table<MAX> tab;
    for (int i = 0; i < a->count;) {
        i = fill<MAX>(a, i, chunk, &tab);
        if (tab.chunks == 0) continue;
        const int blocks = tab.chunks < kBlocks ? tab.chunks : kBlocks;
        const cudaError_t e = launch_early(adamw_kernel<EIGHT, MAX>, blocks, kThreads, 0, stream, tab, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace adamw
}  // namespace gdn

namespace {

using gdn::aligned;
using gdn::fail;

bool finite_from(double v, double least) { return isfinite(v) && v >= least; }

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
    return GDN_OK;
}

}  // namespace

extern "C" gdn_status gdn_adamw(const gdn_adamw_args *a, gdn_stream stream) {
    const gdn_status st = validate(a);
    if (st != GDN_OK) return st;
    gdn::adamw::Step s = {};
    s.beta1 = (float)a->beta1, s.rest1 = (float)(1 - a->beta1);
    s.beta2 = (float)a->beta2, s.rest2 = (float)(1 - a->beta2);
    s.lr = (float)a->lr, s.weight_decay = (float)a->weight_decay, s.eps = (float)a->eps;
    s.max_norm = (float)a->max_norm, s.norm_eps = (float)a->norm_eps;
    // beta = 0 has logarithm -inf, and 1 - beta^t = 1
    s.log_beta1 = (float)log(a->beta1), s.log_beta2 = (float)log(a->beta2);
    if (!a->step_device) {
        s.c1 = (float)-expm1((double)a->step * log(a->beta1));
        s.root2 = (float)sqrt(-expm1((double)a->step * log(a->beta2)));
    }
    s.step = a->step_device, s.lr_at = a->lr_device, s.norm = a->grad_norm, s.err = a->error_word;
    cudaStream_t q = (cudaStream_t)stream;
    const bool eight = a->state_dtype == GDN_DTYPE_E4M3, few = a->count <= gdn::adamw::kFew;
    if (eight)
        return gdn::cuda_status(few ? gdn::adamw::run<true, gdn::adamw::kFew>(a, s, q)
                                    : gdn::adamw::run<true, gdn::adamw::kMany>(a, s, q));
    return gdn::cuda_status(few ? gdn::adamw::run<false, gdn::adamw::kFew>(a, s, q)
                                : gdn::adamw::run<false, gdn::adamw::kMany>(a, s, q));
}
