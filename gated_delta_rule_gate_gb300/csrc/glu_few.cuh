// glu_few.cuh -- the gated feed-forward of few tokens, and the element-wise part of
// its gradient.
//
// Few tokens: bound by the weights' way from HBM.  A warp-level product (m16n8k16) has 8
// rows of w_gate and the same 8 of w_up as its 16 rows, so that a thread's accumulators
// hold gate and up of the same outputs.  The order of k within a product is free: a lane
// takes 8 adjacent values (16 bytes) of its two weight rows and of its token, which are its
// operands of two products over 32 k's.  The block's warps share the k's out and add their
// sums up at the end, in one order.
//
// What counts is bytes on their way: 16 words of 16 bytes a lane, 16 warps an SM, as 16
// features a block and 4 words of each of their rows.  Where that makes less than a block
// an SM (up to 2432 features), 8 features and 8 words.  1 token x 4096, in us:
// features of the call  1536    4864    8192
// 16 a block, 4 words    8.7    14.1    22.1
//  8 a block, 8 words    6.6    14.8    24.8
//  8 a block, 4 words   10.8    15.5    25.8
// The same of more tokens, with weights that L2 does not hold, 16 features a block and 8:
// dim x inner        2048 x 1536  4096 x 2432  4096 x 4864  2048 x 6144  4096 x 8192
// 16 tokens           6.6   4.7   10.6   8.4   15.5  15.6   13.8  12.0   25.8  27.1
// 32 tokens           8.8   6.0   12.5  10.2   16.4  19.0   16.0  15.6   28.3  34.6
// 8 x 4096 x 8192 bf16: 22.4 us, 6.0 TB/s.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "glu_launch.h"
#include "glu_math.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "values.cuh"

namespace gdn {
namespace glu {

constexpr int kFewWarps = 8;

template <typename T>
__device__ __forceinline__ void product16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value) ptx::mma16816(d, a, b0, b1);
    else ptx::mma16816_bf16(d, a, b0, b1);
}
// 8 values of a row of D from k on, zeros beyond it; WORDS: rows are words of 16 bytes.
template <bool WORDS>
__device__ __forceinline__ uint4 load8(const uint16_t *row, int k, int D) {
    if constexpr (WORDS) {
        return k < D ? *reinterpret_cast<const uint4 *>(row + k) : make_uint4(0, 0, 0, 0);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = k + 2 * i < D ? row[k + 2 * i] : 0, hi = k + 2 * i + 1 < D ? row[k + 2 * i + 1] : 0;
            w[i] = lo | hi << 16;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// NT: groups of 8 tokens; MT: of 8 features.
template <typename T, int NT, int MT, bool WORDS>
__global__ void __launch_bounds__(32 * kFewWarps, 2) few_kernel(const __grid_constant__ Few p) {
    constexpr int kAhead = 8 / MT;  // words of a weight row on their way to a lane
    __shared__ float sums[kFewWarps][NT][MT][16][9];
    ptx::grid_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint16_t *wg[MT], *wu[MT], *x[NT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int f = (blockIdx.x * MT + m) * 8 + g, row = f < p.F ? f : p.F - 1;  // those beyond the last are not kept
        wg[m] = static_cast<const uint16_t *>(p.wg) + (int64_t)row * p.D;
        wu[m] = static_cast<const uint16_t *>(p.wu) + (int64_t)row * p.D;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int tok = 8 * n + g;
        x[n] = tok < p.T ? static_cast<const uint16_t *>(p.x) + tok * p.xs : nullptr;
    }
    float acc[NT][MT][4] = {};
    // a warp's steps of 32 k's: kAhead adjacent ones at a time
    const int steps = (p.D + 31) / 32;
    for (int s0 = warp * kAhead; s0 < steps; s0 += kFewWarps * kAhead) {
        uint4 a[MT][kAhead], b[MT][kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int k = (s0 + i) * 32 + 8 * t;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                a[m][i] = load8<WORDS>(wg[m], k, p.D);
                b[m][i] = load8<WORDS>(wu[m], k, p.D);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int k = (s0 + i) * 32 + 8 * t;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 v = x[n] ? load8<WORDS>(x[n], k, p.D) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint32_t first[4] = {a[m][i].x, b[m][i].x, a[m][i].y, b[m][i].y};
                    const uint32_t second[4] = {a[m][i].z, b[m][i].z, a[m][i].w, b[m][i].w};
                    product16<T>(acc[n][m], first, v.x, v.y);
                    product16<T>(acc[n][m], second, v.z, v.w);
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float(&to)[16][9] = sums[warp][n][m];
            to[g][2 * t] = acc[n][m][0], to[g][2 * t + 1] = acc[n][m][1];
            to[8 + g][2 * t] = acc[n][m][2], to[8 + g][2 * t + 1] = acc[n][m][3];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * NT * MT; i += 32 * kFewWarps) {
        const int e = i % (8 * MT), tok = i / (8 * MT), n = tok >> 3, c = tok & 7, at = blockIdx.x * (8 * MT) + e;
        if (tok >= p.T) continue;
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w)
            gate += sums[w][n][e >> 3][e & 7][c], up += sums[w][n][e >> 3][8 + (e & 7)][c];
        if (at < p.F)
            with_activation(p.act, [&](auto act) {
                static_cast<T *>(p.out)[tok * p.os + at] = static_cast<T>(activation<act>(gate) * up);
            });
        if (p.gates && at < p.Fg) {
            unsigned char *row = p.gates + tok * gates_row(p.Fg);
            const uint32_t g = at < p.F ? __float_as_uint(gate) : 0u, u = at < p.F ? __float_as_uint(up) : 0u;
            reinterpret_cast<uint16_t *>(row)[at] = (uint16_t)(g >> 16);
            reinterpret_cast<uint16_t *>(row)[p.Fg + at] = (uint16_t)(u >> 16);
            row[lower_at(p.Fg, 0, at)] = (unsigned char)(g >> 8);
            row[lower_at(p.Fg, 1, at)] = (unsigned char)(u >> 8);
        }
    }
}

template <typename T, int NT, int MT>
cudaError_t launch_few_of(const Few &p, cudaStream_t stream) {
    const unsigned blocks = (unsigned)((p.F + 8 * MT - 1) / (8 * MT));
    return p.words ? launch_early(few_kernel<T, NT, MT, true>, blocks, 32 * kFewWarps, 0, stream, p)
                   : launch_early(few_kernel<T, NT, MT, false>, blocks, 32 * kFewWarps, 0, stream, p);
}
template <typename T>
cudaError_t launch_few(const Few &p, cudaStream_t stream) {
    static_assert(kFewTokens == 32, "groups of 8 tokens");
    const bool narrow = p.F <= 16 * sm_count();
    if (p.T <= 8) return narrow ? launch_few_of<T, 1, 1>(p, stream) : launch_few_of<T, 1, 2>(p, stream);
    if (p.T <= 16) return narrow ? launch_few_of<T, 2, 1>(p, stream) : launch_few_of<T, 2, 2>(p, stream);
    return narrow ? launch_few_of<T, 4, 1>(p, stream) : launch_few_of<T, 4, 2>(p, stream);
}

// ---------------------------------------------------------------- gradient, element by element
// 8 kept values from their upper halves and next bytes.
__device__ __forceinline__ void widen24(uint4 hi, uint2 lo, float (&v)[8]) {
    const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[2] = {lo.x, lo.y};
#pragma unroll
    for (int e = 0; e < 8; ++e)  // bytes: none, the next one, the upper two
        v[e] = __uint_as_float(__byte_perm(h[e >> 1], l[e >> 2], (e & 1 ? 0x3200 : 0x1000) | (4 + (e & 3)) << 4) & 0xffffff00u);
}

// d_g = d_out u act'(g) and d_u = d_out act(g), 8 adjacent values a thread; WORDS: rows of
// d_out are words of 16 bytes (the others are by their making).  Columns from F to Fp
// nobody reads of d_g and d_u.  Bound by HBM: 8192 x 6144 bf16 in 90 us, 6.7 TB/s.
template <typename T, bool WORDS>
__global__ void __launch_bounds__(256) gate_grad_kernel(const __grid_constant__ GateGrad p) {
    ptx::grid_wait();
    const int per = p.Fp / 8;
    const int64_t n = p.rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per;
        const int c = (int)(i - row * per) * 8;
        const T *at = static_cast<const T *>(p.d_out) + row * p.dos + c;
        const unsigned char *gates = p.gates + row * gates_row(p.Fg);
        const uint4 gh = *reinterpret_cast<const uint4 *>(gates + 2 * c);
        const uint4 uh = *reinterpret_cast<const uint4 *>(gates + 2 * (p.Fg + c));
        const uint2 gl = *reinterpret_cast<const uint2 *>(gates + lower_at(p.Fg, 0, c));
        const uint2 ul = *reinterpret_cast<const uint2 *>(gates + lower_at(p.Fg, 1, c));
        float d[8], g[8], u[8], dg[8], du[8];
        if constexpr (WORDS) {
            load_values<T, 8>(at, d);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = c + e < p.F ? static_cast<float>(at[e]) : 0.f;
        }
        widen24(gh, gl, g);
        widen24(uh, ul, u);
        with_activation(p.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 a = activation_slope<act>(g[e]);
                dg[e] = d[e] * u[e] * a.y;
                du[e] = d[e] * a.x;
            }
        });
        store_values<T, 8>(static_cast<T *>(p.dg) + row * p.Fp + c, dg);
        store_values<T, 8>(static_cast<T *>(p.du) + row * p.Fp + c, du);
    }
}
template <typename T>
cudaError_t launch_gate_grad(const GateGrad &p, cudaStream_t stream) {
    const int64_t blocks = (p.rows * (p.Fp / 8) + 255) / 256, most = (int64_t)sm_count() * 16;
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    return p.words ? launch_early(gate_grad_kernel<T, true>, grid, 256, 0, stream, p)
                   : launch_early(gate_grad_kernel<T, false>, grid, 256, 0, stream, p);
}

// ---------------------------------------------------------------- shares of a result
// Four adjacent columns a thread, the shares in their order.
template <typename T>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Joins joins) {
    ptx::grid_wait();
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if (q >= joins.count) break;
        const Join &p = joins.j[q];
        const int per = p.cs / 4;
        const int64_t plane = p.rows * p.cs, n = p.results * p.rows * per;
        for (; i < n; i += (int64_t)gridDim.x * 256) {
            const int64_t line = i / per;  // result and row
            const int c = (int)(i - line * per) * 4, z = line >= p.rows;
            const int64_t row = z ? line - p.rows : line;
            float sum[4] = {};
#pragma unroll 4
            for (int k = 0; k < p.parts; ++k) {
                const float4 v =
                    *reinterpret_cast<const float4 *>(p.shares + (int64_t)k * p.results * plane + line * p.cs + c);
                sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
            }
            T *to = static_cast<T *>(p.out[z]) + row * p.stride + c;
            if (p.words) {
                if (c < p.cols) store_values<T, 4>(to, sum);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < p.cols) to[e] = static_cast<T>(sum[e]);
            }
        }
        i -= n;
    }
}
template <typename T>
cudaError_t launch_join(const Joins &p, cudaStream_t stream) {
    int64_t n = 0;
    for (int q = 0; q < p.count; ++q) n += p.j[q].results * p.j[q].rows * (p.j[q].cs / 4);
    const int64_t blocks = (n + 255) / 256, most = (int64_t)sm_count() * 16;
    return launch_early(join_kernel<T>, (unsigned)(blocks < most ? blocks : most), 256, 0, stream, p);
}

// The same of the forward pass: g and u of four columns, then what the product's kernel
// makes of them.
template <typename T>
__global__ void __launch_bounds__(256) forward_join_kernel(const __grid_constant__ ForwardJoin p) {
    ptx::grid_wait();
    const int per = p.cs / 4;
    const int64_t plane = p.rows * p.cs, n = p.rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per;
        const int c = (int)(i - row * per) * 4;
        float4 g = {}, u = {};
#pragma unroll 4
        for (int k = 0; k < p.parts; ++k) {
            const float *at = p.shares + 2 * k * plane + row * p.cs + c;
            const float4 a = *reinterpret_cast<const float4 *>(at), b = *reinterpret_cast<const float4 *>(at + plane);
            g.x += a.x, g.y += a.y, g.z += a.z, g.w += a.w;
            u.x += b.x, u.y += b.y, u.z += b.z, u.w += b.w;
        }
        const float gs[4] = {g.x, g.y, g.z, g.w}, us[4] = {u.x, u.y, u.z, u.w};
        float v[4];
        with_activation(p.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = activation<act>(gs[e]) * us[e];
        });
        T *to = static_cast<T *>(p.out) + row * p.os + c;
        if (p.words) {
            if (c < p.F) store_values<T, 4>(to, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < p.F) to[e] = static_cast<T>(v[e]);
        }
        if (!p.gates) continue;
        unsigned char *gates = p.gates + row * gates_row(p.Fg);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(k ? us[e] : gs[e]);
            *reinterpret_cast<uint2 *>(gates + 2 * (k * p.Fg + c)) =
                make_uint2(__byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632));
            *reinterpret_cast<uint32_t *>(gates + lower_at(p.Fg, k, c)) =
                __byte_perm(__byte_perm(w[0], w[1], 0x0051), __byte_perm(w[2], w[3], 0x0051), 0x5410);
        }
    }
}
template <typename T>
cudaError_t launch_forward_join(const ForwardJoin &p, cudaStream_t stream) {
    const int64_t blocks = (p.rows * (p.cs / 4) + 255) / 256, most = (int64_t)sm_count() * 16;
    return launch_early(forward_join_kernel<T>, (unsigned)(blocks < most ? blocks : most), 256, 0, stream, p);
}

}  // namespace glu
}  // namespace gdn
