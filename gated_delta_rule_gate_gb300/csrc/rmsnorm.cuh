// rmsnorm.cuh -- gdn_rmsnorm and its gradient: the kernels.
//
// A block takes a row, a thread N groups of V adjacent values of it, which stay in
// registers from the load to the store: every tensor crosses HBM once.  Rows that
// do not fit (more than kFit values) are walked a second time instead.
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

template <typename TA, int V>
__device__ __forceinline__ void load_as(const void *p, bool f32, size_t at, float (&v)[V]) {
    if (f32) load_values<float, V>(static_cast<const float *>(p) + at, v);
    else load_values<TA, V>(static_cast<const TA *>(p) + at, v);
}
template <typename TA, int V>
__device__ __forceinline__ void store_as(void *p, bool f32, size_t at, const float (&v)[V]) {
    if (f32) store_values<float, V>(static_cast<float *>(p) + at, v);
    else store_values<TA, V>(static_cast<TA *>(p) + at, v);
}

template <int V>
__device__ __forceinline__ void store_e4m3(unsigned char *p, const float (&v)[V], float inv) {
    if constexpr (V == 1) {
        *p = __nv_cvt_float_to_fp8(v[0] * inv, __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * inv, v[4 * i + 1] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | hi << 16;
        }
        if constexpr (V == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(p) = w[0];
    }
}
// Scale of a row or group whose largest |y| is m, and its reciprocal.
__device__ __forceinline__ float scale_of(float m, float &inv) {
    m = fmaxf(m, 0x1p-100f);
    inv = kE4m3Max / m;
    return m / kE4m3Max;
}

// Loads r = x + residual of V values at column c.
template <typename TA, int V>
__device__ __forceinline__ void load_r(const Args &p, size_t row, int c, float (&r)[V]) {
    load_values<TA, V>(static_cast<const TA *>(p.x) + row * p.xs + c, r);
    if (p.res) {
        float q[V];
        load_as<TA, V>(p.res, p.res_f32, row * p.D + c, q);
#pragma unroll
        for (int v = 0; v < V; ++v) r[v] += q[v];
    }
}

template <typename TA, int Q, int V, int N>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const __grid_constant__ Args p) {
    ptx::grid_wait();
    __shared__ float s_red[64];
    extern __shared__ int s_peak[];  // V == 1: the largest |y| of each group, as bits
    const size_t row = blockIdx.x;
    const int D = p.D;
    float r[N][V], w[N][V];
    float sum = 0.f, peak = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) r[i][v] = w[i][v] = 0.f;
        if (c < D) {
            load_r<TA, V>(p, row, c, r[i]);
            load_as<TA, V>(p.weight, p.w_f32, c, w[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
        if (p.res_out && c < D) store_as<TA, V>(p.res_out, p.res_f32, row * D + c, r[i]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sum = fmaf(r[i][v], r[i][v], sum);
            if (Q == kRowScale) peak = fmaxf(peak, fabsf(r[i][v] * w[i][v]));
        }
    }
    if (Q == kGroupScale && V == 1) {
        for (int g = threadIdx.x; g < (D + kGroup - 1) / kGroup; g += blockDim.x) s_peak[g] = 0;
    }
    block_sum_max(sum, peak, s_red);
    const float rstd = rsqrtf(sum / (float)D + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) r[i][v] *= rstd * w[i][v];
    if constexpr (Q == kPlain) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
            if (c < D) store_values<TA, V>(static_cast<TA *>(p.out) + row * D + c, r[i]);
        }
    } else if constexpr (Q == kRowScale) {
        float inv;
        const float scale = scale_of(peak * rstd, inv);
        if (threadIdx.x == 0) p.scales[row] = scale;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
            if (c < D) store_e4m3<V>(static_cast<unsigned char *>(p.out) + row * D + c, r[i], inv);
        }
    } else {
        const int groups = (D + kGroup - 1) / kGroup;
        if (V == 1) {
            if (blockDim.x <= 32) __syncwarp();
#pragma unroll
            for (int i = 0; i < N; ++i) {  // 32 adjacent values lie in one group
                const int c = i * (int)blockDim.x + (int)threadIdx.x;
                float m = fabsf(r[i][0]);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                // numbers >= 0 order as their bits; a maximum does not depend on the order
                if ((threadIdx.x & 31) == 0 && c < D) atomicMax(&s_peak[c / kGroup], __float_as_int(m));
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
            float m = 0.f;
            if (V == 1) {
                if (c < D) m = __int_as_float(s_peak[c / kGroup]);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) m = fmaxf(m, fabsf(r[i][v]));
#pragma unroll
                for (int o = kGroup / V / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            }
            float inv;
            const float scale = scale_of(m, inv);
            if (c < D) {
                if (c % kGroup == 0) p.scales[row * groups + c / kGroup] = scale;
                store_e4m3<V>(static_cast<unsigned char *>(p.out) + row * D + c, r[i], inv);
            }
        }
    }
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
        load_r<TA, 1>(p, row, c, r);
        sum = fmaf(r[0], r[0], sum);
        if (Q == kRowScale) {
            load_as<TA, 1>(p.weight, p.w_f32, c, w);
            peak = fmaxf(peak, fabsf(r[0] * w[0]));
        }
    }
    block_sum_max(sum, peak, s_red);
    const float rstd = rsqrtf(sum / (float)D + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
    float inv = 1.f;
    if (Q == kRowScale) {
        const float scale = scale_of(peak * rstd, inv);
        if (threadIdx.x == 0) p.scales[row] = scale;
    }
    // 1024 columns at a time: eight whole groups, four warps each
    for (int base = 0; base < D; base += blockDim.x) {
        const int c = base + threadIdx.x;
        float r[1] = {0.f}, w[1] = {0.f};
        if (c < D) {
            load_r<TA, 1>(p, row, c, r);
            load_as<TA, 1>(p.weight, p.w_f32, c, w);
            if (p.res_out) store_as<TA, 1>(p.res_out, p.res_f32, row * D + c, r);
        }
        float y[1] = {r[0] * (rstd * w[0])};
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
                const float scale = scale_of(m, inv);
                if (c < D && c % kGroup == 0) p.scales[row * ((D + kGroup - 1) / kGroup) + c / kGroup] = scale;
            }
            if (c < D) store_e4m3<1>(static_cast<unsigned char *>(p.out) + row * D + c, y, inv);
        }
    }
}

inline unsigned threads_for(int groups, int n) {
    const int per = (groups + n - 1) / n;
    return (unsigned)((per + 31) / 32 * 32);
}

template <typename TA, int Q>
cudaError_t launch_out(const Args &p, bool vec, cudaStream_t stream) {
    constexpr int V = sizeof(TA) == 4 ? 4 : 8;
    const unsigned rows = (unsigned)p.rows;
    if (vec) {
        const int groups = p.D / V;
        if (groups <= 512) {
            return launch_early(rmsnorm_kernel<TA, Q, V, 1>, rows, threads_for(groups, 1), 0, stream, p);
        }
        if (groups <= 2048) {
            return launch_early(rmsnorm_kernel<TA, Q, V, 2>, rows, threads_for(groups, 2), 0, stream, p);
        }
    }
    const size_t peaks = (size_t)((p.D + kGroup - 1) / kGroup) * sizeof(int);
    if (p.D <= 2048) return launch_early(rmsnorm_kernel<TA, Q, 1, 4>, rows, threads_for(p.D, 4), peaks, stream, p);
    if (p.D <= 8192) return launch_early(rmsnorm_kernel<TA, Q, 1, 8>, rows, threads_for(p.D, 8), peaks, stream, p);
    return launch_early(rmsnorm_wide_kernel<TA, Q>, rows, 1024, 0, stream, p);
}

template <typename TA>
cudaError_t launch_rmsnorm_as(const Args &p, int q, bool vec, cudaStream_t stream) {
    if (q == kPlain) return launch_out<TA, kPlain>(p, vec, stream);
    if (q == kRowScale) return launch_out<TA, kRowScale>(p, vec, stream);
    return launch_out<TA, kGroupScale>(p, vec, stream);
}

// ---------------------------------------------------------------- gradient
// xhat = r rstd, m = mean(weight d_out xhat): dx = rstd (weight d_out - xhat m) +
// d_residual.  A block takes rows b, b + blocks, ...; a thread has the same
// columns of each, so that its share of d_weight stays in registers, and the next
// row's tensors are loaded while this one's sum is formed; the blocks' shares meet in the workspace, which a second kernel adds up in their order.
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
        if (c < D) load_as<TA, V>(p.weight, p.w_f32, c, w[i]);
    }
    // a row's tensors, on their way while the row before is reduced and written (where
    // 64 registers, of blocks of up to 1024 threads, hold both)
    constexpr bool kAhead = V * N <= 4 || (V == 8 && sizeof(TR) == 2);
    struct Row {
        Words<TA, V> d[N];
        Words<TR, V> r[N], g[N];
        float rstd;
    };
    auto fetch = [&](int64_t row, Row &w) {
        if (row >= p.rows) return;
        w.rstd = p.rstd[row];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
            if (c < D) {
                w.d[i].load(static_cast<const TA *>(p.d_out) + row * p.dos + c);
                w.r[i].load(static_cast<const TR *>(p.r) + row * D + c);
                if (p.d_res) w.g[i].load(static_cast<const TR *>(p.d_res) + row * D + c);
            }
        }
    };
    Row next;
#pragma unroll
    for (int i = 0; i < N; ++i) next.d[i].zero(), next.r[i].zero(), next.g[i].zero();
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
            if (c >= D) continue;
            float g[V];
            now.g[i].get(g);  // zeros without d_residual
#pragma unroll
            for (int v = 0; v < V; ++v) g[v] += now.rstd * (d[i][v] - x[i][v] * m);
            store_values<TR, V>(static_cast<TR *>(p.dx) + row * D + c, g);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
        if (c < D) store_values<float, V>(partial + (size_t)blockIdx.x * p.Dp + c, dw[i]);
    }
}

// Rows of up to kNarrow values, a warp each, in pairs of fp32: dx is what is left of
// weight d_out once its part along x is taken away, and of one value or a few that
// can be almost nothing, of which fp32 would keep rounding errors alone.
template <typename TA, typename TR>
__global__ void __launch_bounds__(32) rmsnorm_grad_narrow_kernel(const __grid_constant__ GradArgs p, float *partial) {
    ptx::grid_wait();
    const int c = threadIdx.x;
    const bool on = c < p.D;
    float w[1] = {0.f}, dw = 0.f;
    if (on) load_as<TA, 1>(p.weight, p.w_f32, c, w);
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
        load_as<TA, 1>(p.weight, p.w_f32, c, w);
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
    load_as<TA, 1>(p.weight, p.w_f32, c, w);
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
cudaError_t launch_grad_as(const GradArgs &p, bool vec, int parts, float *ws, cudaStream_t stream) {
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
    if (vec && p.D <= 1024 * V)
        return launch_early(rmsnorm_grad_kernel<TA, TR, V, 1>, grid, threads_for(p.D / V, 1), 0, stream, p, ws);
    if (vec)
        return launch_early(rmsnorm_grad_kernel<TA, TR, V, kTwo>, grid, threads_for(p.D / V, kTwo), 0, stream, p, ws);
    if (p.D <= 2048)
        return launch_early(rmsnorm_grad_kernel<TA, TR, 1, 4>, grid, threads_for(p.D, 4), 0, stream, p, ws);
    return launch_early(rmsnorm_grad_kernel<TA, TR, 1, 8>, grid, threads_for(p.D, 8), 0, stream, p, ws);
}

}  // namespace norm
}  // namespace gdn
