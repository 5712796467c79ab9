// rmsnorm.cuh -- gdn_rmsnorm and its gradient: the kernels.
//
// r = x + residual, y = r rsqrt(mean(r^2) + eps) weight.  A block takes a row, a
// thread N groups of V adjacent values of it, which stay in registers from the load
// to the store: every tensor crosses HBM once, and HBM is the bound.  One row to a
// block needs no loop and no wait between rows; the blocks of an SM overlap one
// another's sums.  The scale of a whole row needs max |r weight| before the row's
// rstd is known, so both reductions are one: |y| is that times rstd >= 0.
// Rows that do not fit (more than kFit values, or 16384 in words of 8) are walked a
// second time instead.
//
// 32768 x 2048 bf16, fp32 residual, e4m3 by groups of 128: 110 us, 6.7 TB/s.
// 256 x 4096 fp16: 5.3 to 8.0 us, with the buffers' places in memory; a launch and two trips
// there.  Rows that do not fit, value by value and read twice: 4096 x 16384 fp32 392 us, where
// HBM would take 129.
#pragma once

#include <cuda_fp8.h>

#include "launch.h"
#include "ptx.cuh"
#include "rmsnorm_launch.h"
#include "twofloat.cuh"
#include "values.cuh"

namespace gdn {
namespace norm {

enum : int { kPlain = 0, kRowScale = 1, kGroupScale = 2 };
constexpr int kGroup = 128;
constexpr float kE4m3Max = 448.f;

// Sums of a and maxima of b over the block; every thread gets both.  `s` is
// shared memory of 64 floats, not in use by another call.
__device__ __forceinline__ void block_sum_max(float &a, float &b, float *s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
    }
    if (warps == 1) return;
    if (lane == 0) s[warp] = a, s[32 + warp] = b;
    __syncthreads();
    a = lane < warps ? s[lane] : 0.f;
    b = lane < warps ? s[32 + lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
    }
}

// Columns c, ... of a row (or the weight) in fp32 or TA.
template <typename TA, int V>
__device__ __forceinline__ void load_as(const void *p, bool f32, size_t row, int c, int n, float (&v)[V]) {
    if (f32) load_columns<float, V>(static_cast<const float *>(p) + row, c, n, v);
    else load_columns<TA, V>(static_cast<const TA *>(p) + row, c, n, v);
}
template <typename TA, int V>
__device__ __forceinline__ void store_as(void *p, bool f32, size_t row, int c, int n, const float (&v)[V]) {
    if (f32) store_columns<float, V>(static_cast<float *>(p) + row, c, n, v);
    else store_columns<TA, V>(static_cast<TA *>(p) + row, c, n, v);
}

__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// Scale of a row or group whose largest |y| is m, and the quotients by it.  y / s itself: a
// product with 1 / s puts values at the edge of two steps on the other one.  A division
// for each value made 32768 x 2048 bf16 with scales by group 115 us, this 110, as the
// product alone: the product's remainder is exact in one fma, and a second one rounds the
// quotient as a division does (Markstein 1990; 1 / s is rounded once, and neither it nor the
// remainder underflows where a step of e4m3 could tell).  The remainder is taken as s q - y,
// so that a y of -0 gives -0.
struct Scale {
    float s, inv, times;
    __device__ __forceinline__ explicit Scale(float m) {
        s = fmaxf(m, 0x1p-100f) / kE4m3Max;
        inv = 1.f / s;
        times = isfinite(s) ? s : 0.f;
    }
    __device__ __forceinline__ float under(float y) const {
        const float q = y * inv;
        return fmaf(fmaf(times, q, -y), -inv, q);
    }
};
// Columns c, ... of a row of n bytes.
template <int V>
__device__ __forceinline__ void store_e4m3(unsigned char *row, int c, int n, const float (&y)[V], const Scale &k) {
    if (c >= n) return;
    if constexpr (V == 1) {
        row[c] = __nv_cvt_float_to_fp8(k.under(y[0]), __NV_SATFINITE, __NV_E4M3);
    } else if constexpr (V == 2) {
        *reinterpret_cast<uint16_t *>(row + c) = (uint16_t)e4m3_pair(k.under(y[0]), k.under(y[1]));
    } else {
        uint32_t w[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            w[i] = e4m3_pair(k.under(y[4 * i]), k.under(y[4 * i + 1])) |
                   e4m3_pair(k.under(y[4 * i + 2]), k.under(y[4 * i + 3])) << 16;
        if constexpr (V == 8) *reinterpret_cast<uint2 *>(row + c) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(row + c) = w[0];
    }
}

// N times V columns of a row in fp32 or TA, all on their way before the first is
// looked at; `column(i)` gives the i-th's first.
template <typename TA, int V, int N, typename C>
__device__ __forceinline__ void load_row(const void *p, bool f32, size_t row, int n, C column, float (&v)[N][V]) {
    if (f32) {
        Columns<float, V> q[N];
        const float *r = static_cast<const float *>(p) + row;
#pragma unroll
        for (int i = 0; i < N; ++i) q[i].load(r, column(i), n);
#pragma unroll
        for (int i = 0; i < N; ++i) q[i].get(v[i]);
    } else {
        Columns<TA, V> q[N];
        const TA *r = static_cast<const TA *>(p) + row;
#pragma unroll
        for (int i = 0; i < N; ++i) q[i].load(r, column(i), n);
#pragma unroll
        for (int i = 0; i < N; ++i) q[i].get(v[i]);
    }
}
// r = x + residual.
template <typename TA, int V, int N, typename C>
__device__ __forceinline__ void load_sum(const Args &p, size_t row, C column, float (&v)[N][V]) {
    Columns<TA, V> x[N];
    const TA *r = static_cast<const TA *>(p.x) + row * p.xs;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i].load(r, column(i), p.D);
    float q[N][V];
    if (p.res) {
        load_row<TA, V, N>(p.res, p.res_f32, row * p.D, p.D, column, q);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) q[i][k] = -0.f;  // x + -0 is x, of either zero
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i].get(v[i]);
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][k] += q[i][k];
    }
}

// V: 8 or 4, words of 16 bytes; 2, rows whose values pair up; 1, rows at any alignment.
// 16384 rows of bf16 with a residual and scales by group: 2048 wide (V = 8) 46 us,
// 2046 (V = 2) 85, against 143 by single values; 2047 (V = 1) 129; fp32 74, 81, 125.
// Eight values a thread at every V: four at V = 1 took 142 us, with fewer bytes on
// their way.  Rows of up to 512 words take one a thread and four blocks an SM at 32
// registers; longer ones two.
template <typename TA, int Q, int V, int N>
__global__ void __launch_bounds__(V > 2 && N == 1 ? 512 : 1024, V > 2 && N == 1 ? 4 : 1)
    rmsnorm_kernel(const __grid_constant__ Args p) {
    __shared__ float s_red[64];
    extern __shared__ int s_peak[];  // V <= 2: the largest |y| of each group, as bits
    ptx::grid_wait();
    const size_t row = blockIdx.x;
    const int D = p.D;
    auto column = [&](int i) { return (i * (int)blockDim.x + (int)threadIdx.x) * V; };
    float r[N][V];
    float sum = 0.f, peak = 0.f;
    load_sum<TA, V, N>(p, row, column, r);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (p.res_out) store_as<TA, V>(p.res_out, p.res_f32, row * D, column(i), D, r[i]);
#pragma unroll
        for (int v = 0; v < V; ++v) sum = fmaf(r[i][v], r[i][v], sum);
    }
    if (Q == kRowScale) {
        float w[N][V];
        load_row<TA, V, N>(p.weight, p.w_f32, 0, D, column, w);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) peak = fmaxf(peak, fabsf(r[i][v] * w[i][v]));
    }
    if (Q == kGroupScale && V <= 2) {
        for (int g = threadIdx.x; g < (D + kGroup - 1) / kGroup; g += blockDim.x) s_peak[g] = 0;
    }
    block_sum_max(sum, peak, s_red);
    const float rstd = rsqrtf(sum / (float)D + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
    {
        float w[N][V];
        load_row<TA, V, N>(p.weight, p.w_f32, 0, D, column, w);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) r[i][v] = r[i][v] * rstd * w[i][v];
    }
    unsigned char *bytes = static_cast<unsigned char *>(p.out) + row * D;
    if constexpr (Q == kPlain) {
#pragma unroll
        for (int i = 0; i < N; ++i) store_columns<TA, V>(static_cast<TA *>(p.out) + row * D, column(i), D, r[i]);
    } else if constexpr (Q == kRowScale) {
        const Scale scale(peak * rstd);
        if (threadIdx.x == 0) p.scales[row] = scale.s;
#pragma unroll
        for (int i = 0; i < N; ++i) store_e4m3<V>(bytes, column(i), D, r[i], scale);
    } else {
        const int groups = (D + kGroup - 1) / kGroup;
        float m[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            m[i] = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) m[i] = fmaxf(m[i], fabsf(r[i][v]));
            // of whole words the lanes of a group are part of a warp
            constexpr int kLanes = V <= 2 ? 32 : kGroup / V;
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
        }
        if (V <= 2) {
            if (blockDim.x <= 32) __syncwarp();
#pragma unroll
            for (int i = 0; i < N; ++i) {  // a warp's columns lie in one group
                // numbers >= 0 order as their bits; a maximum does not depend on the order
                if ((threadIdx.x & 31) == 0 && column(i) < D)
                    atomicMax(&s_peak[column(i) / kGroup], __float_as_int(m[i]));
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i) m[i] = column(i) < D ? __int_as_float(s_peak[column(i) / kGroup]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = column(i);
            const Scale scale(m[i]);
            if (c < D && c % kGroup == 0) p.scales[row * groups + c / kGroup] = scale.s;
            store_e4m3<V>(bytes, c, D, r[i], scale);
        }
    }
}

template <typename TA>
__device__ __forceinline__ float sum_at(const Args &p, size_t row, int c) {
    float r = static_cast<float>(static_cast<const TA *>(p.x)[row * p.xs + c]), q[1];
    if (!p.res) return r;
    load_as<TA, 1>(p.res, p.res_f32, row * p.D, c, p.D, q);
    return r + q[0];
}

// Rows that do not fit in registers: x and residual are read again.  The second
// walk is also the one that writes, so that residual_out may be residual.
template <typename TA, int Q>
__global__ void __launch_bounds__(1024) rmsnorm_wide_kernel(const __grid_constant__ Args p) {
    ptx::grid_wait();
    __shared__ float s_red[64], s_group[64];
    const size_t row = blockIdx.x;
    const int D = p.D;
    float sum = 0.f, peak = 0.f;
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
        float r[1], w[1];
        r[0] = sum_at<TA>(p, row, c);
        sum = fmaf(r[0], r[0], sum);
        if (Q == kRowScale) {
            load_as<TA, 1>(p.weight, p.w_f32, 0, c, D, w);
            peak = fmaxf(peak, fabsf(r[0] * w[0]));
        }
    }
    block_sum_max(sum, peak, s_red);
    const float rstd = rsqrtf(sum / (float)D + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
    Scale scale(peak * rstd);
    if (Q == kRowScale && threadIdx.x == 0) p.scales[row] = scale.s;
    // 1024 columns at a time: eight whole groups, four warps each
    for (int base = 0; base < D; base += blockDim.x) {
        const int c = base + threadIdx.x;
        float r[1] = {0.f}, w[1] = {0.f};
        if (c < D) {
            r[0] = sum_at<TA>(p, row, c);
            load_as<TA, 1>(p.weight, p.w_f32, 0, c, D, w);
            if (p.res_out) store_as<TA, 1>(p.res_out, p.res_f32, row * D, c, D, r);
        }
        float y[1] = {r[0] * rstd * w[0]};
        if constexpr (Q == kPlain) {
            if (c < D) store_values<TA, 1>(static_cast<TA *>(p.out) + row * D + c, y);
        } else {
            if (Q == kGroupScale) {
                float m = fabsf(y[0]);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                __syncthreads();
                if ((threadIdx.x & 31) == 0) s_group[threadIdx.x >> 5] = m;
                __syncthreads();
                const int g = threadIdx.x >> 7;
                m = fmaxf(fmaxf(s_group[4 * g], s_group[4 * g + 1]), fmaxf(s_group[4 * g + 2], s_group[4 * g + 3]));
                scale = Scale(m);
                if (c < D && c % kGroup == 0) p.scales[row * ((D + kGroup - 1) / kGroup) + c / kGroup] = scale.s;
            }
            store_e4m3<1>(static_cast<unsigned char *>(p.out) + row * D, c, D, y, scale);
        }
    }
}

inline unsigned threads_for(int groups, int n) {
    const int per = (groups + n - 1) / n;
    return (unsigned)((per + 31) / 32 * 32);
}

template <typename TA, int Q>
cudaError_t launch_out(const Args &p, int width, cudaStream_t stream) {
    constexpr int V = sizeof(TA) == 4 ? 4 : 8;
    const unsigned rows = (unsigned)p.rows;
    if (width == V) {
        const int groups = p.D / V;
        if (groups <= 512) {
            return launch_early(rmsnorm_kernel<TA, Q, V, 1>, rows, threads_for(groups, 1), 0, stream, p);
        }
        if (groups <= 2048) {
            return launch_early(rmsnorm_kernel<TA, Q, V, 2>, rows, threads_for(groups, 2), 0, stream, p);
        }
    }
    const size_t peaks = (size_t)((p.D + kGroup - 1) / kGroup) * sizeof(int);
    if (p.D <= kFit && width >= 2)
        return launch_early(rmsnorm_kernel<TA, Q, 2, 4>, rows, threads_for(p.D / 2, 4), peaks, stream, p);
    if (p.D <= kFit) return launch_early(rmsnorm_kernel<TA, Q, 1, 8>, rows, threads_for(p.D, 8), peaks, stream, p);
    return launch_early(rmsnorm_wide_kernel<TA, Q>, rows, 1024, 0, stream, p);
}

template <typename TA>
cudaError_t launch_rmsnorm_as(const Args &p, int q, int width, cudaStream_t stream) {
    if (q == kPlain) return launch_out<TA, kPlain>(p, width, stream);
    if (q == kRowScale) return launch_out<TA, kRowScale>(p, width, stream);
    return launch_out<TA, kGroupScale>(p, width, stream);
}

// ---------------------------------------------------------------- gradient
// xhat = r rstd, m = mean(weight d_out xhat): dx = rstd (weight d_out - xhat m) +
// d_residual, d_weight = sum of d_out xhat over the rows.  A block takes rows b, b +
// blocks, ...; a thread has the same columns of each, so that its share of d_weight
// stays in registers, and the next row's tensors are loaded while this one's sum is
// formed.  The blocks' shares meet in the workspace, and a second kernel adds them up
// in their order: no atomics, the same sum every time.
//
// Bound by HBM, and by the wait for each row's sum: forward and gradient of 32768 x
// 2048 bf16 181 us, 5.2 TB/s; of 16384 x 2046 by pairs 122 against 206 by single values,
// 16384 x 2048 96.  Wide rows take two kernels, value by value, that read everything twice:
// 4096 x 16384 fp32 with its forward 689 us, where HBM would take 277.
template <typename TA, typename TR, int V, int N>
__global__ void __launch_bounds__(1024) rmsnorm_grad_kernel(const __grid_constant__ GradArgs p, float *partial) {
    ptx::grid_wait();
    __shared__ float s_red[2][64];
    const int D = p.D;
    float w[N][V], dw[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) w[i][v] = dw[i][v] = 0.f;
        load_as<TA, V>(p.weight, p.w_f32, 0, c, D, w[i]);
    }
    // a row's tensors, on their way while the row before is reduced and written (where
    // 64 registers, of blocks of up to 1024 threads, hold both)
    constexpr bool kAhead = V * N <= 4 || (V == 8 && sizeof(TR) == 2);
    struct Row {
        Columns<TA, V> d[N];
        Columns<TR, V> r[N], g[N];
        float rstd;
    };
    auto fetch = [&](int64_t row, Row &w) {
        if (row >= p.rows) return;
        w.rstd = p.rstd[row];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
            w.d[i].load(static_cast<const TA *>(p.d_out) + row * p.dos, c, D);
            w.r[i].load(static_cast<const TR *>(p.r) + row * D, c, D);
            if (p.d_res) w.g[i].load(static_cast<const TR *>(p.d_res) + row * D, c, D);
        }
    };
    Row next;
    if (kAhead) fetch(blockIdx.x, next);
    int par = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
        if (!kAhead) fetch(row, next);
        const Row now = next;
        if (kAhead) fetch(row + gridDim.x, next);
        float d[N][V], x[N][V];
        float dot = 0.f, none = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
            now.d[i].get(d[i]);
            now.r[i].get(x[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[i][v] *= now.rstd;
                dw[i][v] = fmaf(d[i][v], x[i][v], dw[i][v]);
                d[i][v] *= w[i][v];
                dot = fmaf(d[i][v], x[i][v], dot);
            }
        }
        block_sum_max(dot, none, s_red[par]);
        const float m = dot / (float)D;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
            float g[V] = {};
            if (p.d_res) now.g[i].get(g);
#pragma unroll
            for (int v = 0; v < V; ++v) g[v] += now.rstd * (d[i][v] - x[i][v] * m);
            store_columns<TR, V>(static_cast<TR *>(p.dx) + row * D, c, D, g);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
        store_columns<float, V>(partial + (size_t)blockIdx.x * p.Dp, c, D, dw[i]);
    }
}

// Rows of up to kNarrow values, a warp each, in pairs of fp32: dx is what is left of
// weight d_out once its part along x is taken away, and of one value or a few that
// can be almost nothing, of which fp32 would keep rounding errors alone.  It is then the
// gradient for the rstd that is given, whose own rounding, up to 2^-22, is up to
// 2^-22 (1 + 3 sqrt(D)) rstd |weight d_out| of it: more than dx itself where D is 1 and r^2 far
// above eps.
template <typename TA, typename TR>
__global__ void __launch_bounds__(32) rmsnorm_grad_narrow_kernel(const __grid_constant__ GradArgs p, float *partial) {
    ptx::grid_wait();
    const int c = threadIdx.x;
    const bool on = c < p.D;
    float w[1] = {0.f}, dw = 0.f;
    load_as<TA, 1>(p.weight, p.w_f32, 0, c, p.D, w);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float rstd = p.rstd[row];
        float d = 0.f, r = 0.f;
        if (on) {
            d = static_cast<float>(static_cast<const TA *>(p.d_out)[row * p.dos + c]);
            r = static_cast<float>(static_cast<const TR *>(p.r)[row * p.D + c]);
        }
        const TwoFloat x = two_product(r, rstd), wd = two_product(d, w[0]);
        dw = fmaf(d, x.hi, dw);
        const TwoFloat m = warp_sum(wd * x) / (float)p.D, g = TwoFloat{rstd, 0.f} * (wd + -(x * m));
        float res = 0.f;
        if (on && p.d_res) res = static_cast<float>(static_cast<const TR *>(p.d_res)[row * p.D + c]);
        if (on) static_cast<TR *>(p.dx)[row * p.D + c] = static_cast<TR>(g.hi + res);
    }
    if (on) partial[(size_t)blockIdx.x * p.Dp + c] = dw;
}

// Wide rows: the mean of each row first, then columns over a stretch of rows.
template <typename TA, typename TR>
__global__ void __launch_bounds__(1024) rmsnorm_grad_mean_kernel(const __grid_constant__ GradArgs p, float *mean) {
    ptx::grid_wait();
    __shared__ float s_red[64];
    const int64_t row = blockIdx.x;
    float dot = 0.f, none = 0.f;
    const float rstd = p.rstd[row];
    for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
        float w[1];
        load_as<TA, 1>(p.weight, p.w_f32, 0, c, p.D, w);
        const float d = static_cast<float>(static_cast<const TA *>(p.d_out)[row * p.dos + c]);
        const float r = static_cast<float>(static_cast<const TR *>(p.r)[row * p.D + c]);
        dot = fmaf(d * w[0], r * rstd, dot);
    }
    block_sum_max(dot, none, s_red);
    if (threadIdx.x == 0) mean[row] = dot / (float)p.D;
}
template <typename TA, typename TR>
__global__ void __launch_bounds__(256) rmsnorm_grad_columns_kernel(const __grid_constant__ GradArgs p,
                                                                  const float *mean, float *partial, int column_blocks) {
    ptx::grid_wait();
    const int c = (int)(blockIdx.x % column_blocks) * 256 + (int)threadIdx.x;
    const int part = blockIdx.x / column_blocks, parts = gridDim.x / column_blocks;
    if (c >= p.D) return;
    float w[1], dw = 0.f;
    load_as<TA, 1>(p.weight, p.w_f32, 0, c, p.D, w);
    for (int64_t row = part; row < p.rows; row += parts) {
        const float rstd = p.rstd[row], m = mean[row];
        const float d = static_cast<float>(static_cast<const TA *>(p.d_out)[row * p.dos + c]);
        const float x = static_cast<float>(static_cast<const TR *>(p.r)[row * p.D + c]) * rstd;
        float g = p.d_res ? static_cast<float>(static_cast<const TR *>(p.d_res)[row * p.D + c]) : 0.f;
        dw = fmaf(d, x, dw);
        g += rstd * (d * w[0] - x * m);
        static_cast<TR *>(p.dx)[row * p.D + c] = static_cast<TR>(g);
    }
    partial[(size_t)part * p.Dp + c] = dw;
}

template <typename TA, typename TR>
cudaError_t launch_grad_as(const GradArgs &p, int width, int parts, float *ws, cudaStream_t stream) {
    constexpr int V = sizeof(TA) == 4 || sizeof(TR) == 4 ? 4 : 8;
    const unsigned grid = (unsigned)parts;
    if (p.D > kFit) {
        float *mean = ws + (size_t)parts * p.Dp;
        const cudaError_t e =
            launch_early(rmsnorm_grad_mean_kernel<TA, TR>, (unsigned)p.rows, 1024, 0, stream, p, mean);
        if (e != cudaSuccess) return e;
        const int cb = (p.D + 255) / 256;
        return launch_early(rmsnorm_grad_columns_kernel<TA, TR>, grid * cb, 256, 0, stream, p, mean, ws, cb);
    }
    if (p.D <= kNarrow) return launch_early(rmsnorm_grad_narrow_kernel<TA, TR>, grid, 32, 0, stream, p, ws);
    constexpr int kTwo = kFit / 1024 / V;
    if (width == V && p.D <= 1024 * V)
        return launch_early(rmsnorm_grad_kernel<TA, TR, V, 1>, grid, threads_for(p.D / V, 1), 0, stream, p, ws);
    if (width == V)
        return launch_early(rmsnorm_grad_kernel<TA, TR, V, kTwo>, grid, threads_for(p.D / V, kTwo), 0, stream, p, ws);
    if (width == 2 && p.D <= 2048)
        return launch_early(rmsnorm_grad_kernel<TA, TR, 2, 2>, grid, threads_for(p.D / 2, 2), 0, stream, p, ws);
    if (width == 2)
        return launch_early(rmsnorm_grad_kernel<TA, TR, 2, 4>, grid, threads_for(p.D / 2, 4), 0, stream, p, ws);
    if (p.D <= 2048) return launch_early(rmsnorm_grad_kernel<TA, TR, 1, 4>, grid, threads_for(p.D, 4), 0, stream, p, ws);
    return launch_early(rmsnorm_grad_kernel<TA, TR, 1, 8>, grid, threads_for(p.D, 8), 0, stream, p, ws);
}

}  // namespace norm
}  // namespace gdn
