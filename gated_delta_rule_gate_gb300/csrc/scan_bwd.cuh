// scan_bwd.cuh -- gdn_scan_backward: the gradient of the gated linear
// recurrence, parallel over channels and along time, in one launch.
//
// With dh the gradient that reaches h_t and c = a_{t+1} dh_{t+1} what the next
// token hands back (at a request's last token the gradient of its final state):
//     dh = d_o + c,   dx = n i dh,   di = n x dh,   dg = a h_{t-1} dh + n'(g) i x dh
// and in the raw arm d_decay = dg scale sigmoid(z), d_bias = sum of d_decay,
// d_scale = sum of dg softplus(z), z = decay + bias.  c is again a composition of affine maps, from the
// right: a run of tokens takes c to A c + C, with the product A of the forward
// run.  h_{t-1} is formed anew from the state that the forward pass kept before
// every 64th token: a block's tile is 64 tokens, so the forward runs meet in the
// block alone, and only c crosses blocks (one cluster barrier a window, as in the
// forward pass).  x, decay, beta and d_o cross HBM once.  The sums over tokens are
// kept in registers by channel and joined in a fixed order at the end.
#pragma once

#include "scan_cluster.cuh"

namespace gdn {
namespace scan {

__device__ __forceinline__ void gradient_duties(const GradArgs &q, int warps, int warp, int lane, int c, bool report) {
    const Args &p = q.f;
    for (int b = warp; b < p.B; b += warps) {
        int t0, t1;
        request_tokens(p, b, t0, t1);
        const int row = request_row(p, b);
        if (report && lane == 0 && p.err) {
            if (row < 0) atomicOr(p.err, kErrBadSlot);
            if (p.cu && clamped_offset(p, b + 1) < clamped_offset(p, b)) atomicOr(p.err, kErrOverlap);
        }
        if (t0 == t1 && row >= 0 && q.dinit) {
            const size_t at = (size_t)row * p.D;
            store_state(q.dinit + at, c, p.D, q.dfin ? load_state(q.dfin + at, c, p.D) : make_float2(0.f, 0.f));
        }
    }
}

template <typename TA, typename TG, bool RAW, bool BETA>
struct Backward {
    static constexpr int kTokens = 8;
    static constexpr int kTile = kWarps * kTokens;
    static_assert(kTile == kChunk, "a tile begins where the forward pass kept a state");

    struct Raw {
        pair_t<TA> x[kTokens], d[kTokens];
        pair_t<TG> z[kTokens], y[BETA ? kTokens : 1];
    };

    static __device__ __forceinline__ void load(const GradArgs &q, int t, int c, unsigned own, Raw &r) {
        const Args &p = q.f;
        const TA *x = static_cast<const TA *>(p.x) + (int64_t)t * p.xs + c;
        const TA *d = static_cast<const TA *>(q.d_o) + (int64_t)t * q.dos + c;
        const TG *z = static_cast<const TG *>(p.decay) + (int64_t)t * p.gs + c;
        const TG *y = BETA ? static_cast<const TG *>(p.beta) + (int64_t)t * p.bs + c : nullptr;
        const bool vec = p.vec, ok1 = c + 1 < p.D;
        if (c >= p.D) own = 0u;
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            const bool on = own >> k & 1u;
            r.x[k] = on ? load_pair<TA>(x + k * p.xs, vec, ok1) : zero_pair<TA>();
            r.d[k] = on ? load_pair<TA>(d + k * q.dos, vec, ok1) : zero_pair<TA>();
            r.z[k] = on ? load_pair<TG>(z + k * p.gs, vec, ok1) : zero_pair<TG>();
            if (BETA) r.y[k] = on ? load_pair<TG>(y + k * p.bs, vec, ok1) : zero_pair<TG>();
        }
    }

    struct Sums {
        float2 bias, scale;
    };

    template <int MODE>
    static __device__ __forceinline__ void run(const GradArgs &q, Sums &sums) {
        __shared__ float4 s_fwd[2][kWarps][32];  // (A, H) of each warp's run
        __shared__ float2 s_rev[2][kWarps][32];  // C of each warp's run
        __shared__ float4 s_rank[2][kMaxCluster][32];
        const Args &p = q.f;
        const int S = cluster_size(), rank = cluster_rank();
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int c = (int)(blockIdx.x / S) * 64 + 2 * lane;
        const bool ok0 = c < p.D, ok1 = c + 1 < p.D;
        if (S > 1) cluster_arrive();  // waited for before the first remote store
        gradient_duties(q, S * kWarps, rank * kWarps + warp, lane, c, blockIdx.x < S);
        float2 bias = make_float2(0.f, 0.f), scale = bias;
        if (RAW) bias = load_state(p.bias, c, p.D), scale = load_state(p.scale, c, p.D);
        if (S > 1) cluster_wait();

        const int window = S * kTile, steps = (p.T + window - 1) / window;
        Seen seen;
        float2 carry = make_float2(0.f, 0.f);  // c behind the window
        for (int step = steps - 1; step >= 0; --step) {
            const int par = step & 1;
            const int tile = step * window + rank * kTile, t = tile + warp * kTokens;
            const Tokens tok = look_up(p, t, kTokens, lane, seen);
            Raw raw;
            load(q, t, c, tok.own, raw);
            float2 h = make_float2(0.f, 0.f);
            if (tile < p.T) h = load_state(p.chunk + (size_t)(tile / kChunk) * p.D, c, p.D);

            float2 a[kTokens], u[kTokens];
            float4 fwd = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
            for (int k = 0; k < kTokens; ++k) {
                a[k] = make_float2(1.f, 1.f), u[k] = make_float2(0.f, 0.f);
                if (tok.own >> k & 1u) {
                    const float2 z = unpack<TG>(raw.z[k]), y = BETA ? unpack<TG>(raw.y[k]) : z;
                    const float2 x = unpack<TA>(raw.x[k]);
                    const Terms t0 = gate_terms<RAW, BETA, MODE>(z.x, y.x, bias.x, scale.x, p.sigmoid);
                    const Terms t1 = gate_terms<RAW, BETA, MODE>(z.y, y.y, bias.y, scale.y, p.sigmoid);
                    a[k] = make_float2(t0.a, t1.a);
                    u[k] = make_float2(t0.n * t0.i * x.x, t1.n * t1.i * x.y);
                }
                if (tok.first >> k & 1u) {
                    const float2 h0 = first_state(p, tok, k, c);
                    fwd.y = fmaf(a[k].x, h0.x, u[k].x);
                    fwd.w = fmaf(a[k].y, h0.y, u[k].y);
                } else {
                    fwd.y = fmaf(a[k].x, fwd.y, u[k].x);
                    fwd.w = fmaf(a[k].y, fwd.w, u[k].y);
                    fwd.x *= a[k].x;
                    fwd.z *= a[k].y;
                }
            }
            float2 rev = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = kTokens - 1; k >= 0; --k) {
                float2 d = unpack<TA>(raw.d[k]);
                if (tok.last >> k & 1u) add_final(q, tok, k, c, d);
                rev = make_float2(a[k].x * (d.x + rev.x), a[k].y * (d.y + rev.y));
                if (tok.first >> k & 1u) rev = make_float2(0.f, 0.f);
            }
            if (tok.first) fwd.x = fwd.z = kBegins;
            s_fwd[par][warp][lane] = fwd;
            s_rev[par][warp][lane] = rev;
            __syncthreads();
            for (int w = 0; w < warp; ++w) h = apply(s_fwd[par][w][lane], h);
            float4 after = make_float4(1.f, 0.f, 1.f, 0.f), whole = after;
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                if (w == warp) after = whole;
                const float4 f = s_fwd[par][w][lane];
                const float2 r = s_rev[par][w][lane];
                fold(whole, make_float4(f.x, r.x, f.z, r.y));
            }
            float2 dc = carry;
            if (S > 1) {
                for (int r = warp; r < S; r += kWarps) store_remote(&s_rank[par][rank][lane], r, whole);
                cluster_arrive();
                cluster_wait();
                for (int r = S - 1; r >= 0; --r) {
                    if (r == rank) dc = carry;
                    carry = apply(s_rank[par][r][lane], carry);
                }
            } else {
                carry = apply(whole, carry);
            }
            dc = apply(after, dc);

            float2 prev[kTokens];
#pragma unroll
            for (int k = 0; k < kTokens; ++k) {
                if (tok.first >> k & 1u) h = first_state(p, tok, k, c);
                prev[k] = h;
                h = make_float2(fmaf(a[k].x, h.x, u[k].x), fmaf(a[k].y, h.y, u[k].y));
            }
            TA *dx = static_cast<TA *>(q.dx) + (int64_t)t * q.dxs + c;
            TG *dg = static_cast<TG *>(q.dg) + (int64_t)t * q.dgs + c;
            TG *db = BETA ? static_cast<TG *>(q.db) + (int64_t)t * q.dbs + c : nullptr;
#pragma unroll
            for (int k = kTokens - 1; k >= 0; --k) {
                if (!(tok.own >> k & 1u)) continue;  // hands c on
                float2 dh = unpack<TA>(raw.d[k]);
                if (tok.last >> k & 1u) add_final(q, tok, k, c, dh);
                dh.x += dc.x;
                dh.y += dc.y;
                const float2 z = unpack<TG>(raw.z[k]), y = BETA ? unpack<TG>(raw.y[k]) : z;
                const float2 x = unpack<TA>(raw.x[k]);
                const Terms t0 = gate_terms<RAW, BETA, MODE>(z.x, y.x, bias.x, scale.x, p.sigmoid);
                const Terms t1 = gate_terms<RAW, BETA, MODE>(z.y, y.y, bias.y, scale.y, p.sigmoid);
                dc = make_float2(t0.a * dh.x, t1.a * dh.y);
                float g0 = dc.x * prev[k].x, g1 = dc.y * prev[k].y;
                if (MODE != kNone) {
                    g0 = fmaf(t0.dn * t0.i * x.x, dh.x, g0);
                    g1 = fmaf(t1.dn * t1.i * x.y, dh.y, g1);
                }
                if (RAW) {
                    sums.scale.x = fmaf(g0, t0.soft, sums.scale.x);
                    sums.scale.y = fmaf(g1, t1.soft, sums.scale.y);
                    g0 *= t0.dgdz;
                    g1 *= t1.dgdz;
                    sums.bias.x += g0;
                    sums.bias.y += g1;
                }
                if (ok0) {
                    store_pair<TA>(dx + k * q.dxs, make_float2(t0.n * t0.i * dh.x, t1.n * t1.i * dh.y), p.vec, ok1);
                    store_pair<TG>(dg + k * q.dgs, make_float2(g0, g1), p.vec, ok1);
                    if (BETA)
                        store_pair<TG>(db + k * q.dbs,
                                       make_float2(t0.n * x.x * dh.x * t0.di, t1.n * x.y * dh.y * t1.di), p.vec, ok1);
                }
                if (tok.first >> k & 1u) {
                    const int row = __shfl_sync(0xffffffffu, tok.row, k);
                    if (q.dinit) store_state(q.dinit + (size_t)row * p.D, c, p.D, dc);
                    dc = make_float2(0.f, 0.f);
                }
            }
        }
        if (RAW) {  // sums over the block's warps, then over the cluster's blocks
            __syncthreads();
            s_fwd[0][warp][lane] = make_float4(sums.bias.x, sums.bias.y, sums.scale.x, sums.scale.y);
            __syncthreads();
            if (warp == 0) {
                float4 v = s_fwd[0][0][lane];
                for (int w = 1; w < kWarps; ++w) {
                    const float4 o = s_fwd[0][w][lane];
                    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                }
                // the buffer that the last window did not use; no block writes it any more
                if (S > 1) store_remote(&s_rank[1][rank][lane], 0, v);
                else s_rank[1][0][lane] = v;
            }
            if (S > 1) {
                cluster_arrive();
                cluster_wait();
            }
            if (rank == 0 && warp == 0) {
                float4 v = s_rank[1][0][lane];
                for (int r = 1; r < S; ++r) {
                    const float4 o = s_rank[1][r][lane];
                    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                }
                if (q.dbias) store_state(q.dbias, c, p.D, make_float2(v.x, v.y));
                if (q.dscale) store_state(q.dscale, c, p.D, make_float2(v.z, v.w));
            }
        }
    }

    static __device__ __forceinline__ float2 first_state(const Args &p, const Tokens &tok, int k, int c) {
        const int row = __shfl_sync(0xffffffffu, tok.row, k);
        return p.init ? load_state(p.init + (size_t)row * p.D, c, p.D) : make_float2(0.f, 0.f);
    }
    static __device__ __forceinline__ void add_final(const GradArgs &q, const Tokens &tok, int k, int c, float2 &d) {
        const int row = __shfl_sync(0xffffffffu, tok.row, k);
        if (!q.dfin) return;
        const float2 f = load_state(q.dfin + (size_t)row * q.f.D, c, q.f.D);
        d.x += f.x;
        d.y += f.y;
    }
};

template <typename TA, typename TG, bool RAW, bool BETA, int MODE>
__global__ void __launch_bounds__(kWarps * 32, 2) scan_grad_kernel(const __grid_constant__ GradArgs q) {
    typename Backward<TA, TG, RAW, BETA>::Sums sums = {};
    Backward<TA, TG, RAW, BETA>::template run<MODE>(q, sums);
}

template <typename TA, typename TG, bool RAW, bool BETA, int MODE>
cudaError_t launch_grad_one(const GradArgs &q, cudaStream_t stream) {
    auto kernel = scan_grad_kernel<TA, TG, RAW, BETA, MODE>;
    int per_sm = 1;
    cudaError_t e = blocks_per_sm((const void *)kernel, kWarps * 32, 0, &per_sm);
    if (e == cudaSuccess) e = large_clusters((const void *)kernel);
    if (e != cudaSuccess) return e;
    const int cb = (q.f.D + 63) / 64, tile = Backward<TA, TG, RAW, BETA>::kTile;
    const int S = cluster_blocks(cb, (q.f.T + tile - 1) / tile, per_sm * sm_count());
    return launch_clusters(kernel, q, cb, S, stream);
}

template <typename TA, typename TG, bool RAW, bool BETA>
cudaError_t launch_grad_mode(const GradArgs &q, cudaStream_t stream) {
    if (q.f.mode == kNone) return launch_grad_one<TA, TG, RAW, BETA, kNone>(q, stream);
    if (q.f.mode == kLerp) return launch_grad_one<TA, TG, RAW, BETA, kLerp>(q, stream);
    return launch_grad_one<TA, TG, RAW, BETA, kUnit>(q, stream);
}

template <typename TA, typename TG>
cudaError_t launch_grad_types(const GradArgs &q, cudaStream_t stream) {
    if (q.f.bias)
        return q.f.beta ? launch_grad_mode<TA, TG, true, true>(q, stream)
                        : launch_grad_mode<TA, TG, true, false>(q, stream);
    return q.f.beta ? launch_grad_mode<TA, TG, false, true>(q, stream)
                    : launch_grad_mode<TA, TG, false, false>(q, stream);
}

}  // namespace scan
}  // namespace gdn
