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
// block alone, and only c crosses blocks (one exchange a window, as in the
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
        __shared__ float2 s_fwd[kWarps][64];  // (A, H) of each warp's run; at the end its sums
        __shared__ Meeting s_rev;
        __shared__ Exchange s_x;
        const Args &p = q.f;
        const int S = cluster_size(), rank = cluster_rank();
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int c = (int)(blockIdx.x / S) * 64 + 2 * lane;
        const bool ok0 = c < p.D, ok1 = c + 1 < p.D;
        gradient_duties(q, S * kWarps, rank * kWarps + warp, lane, c, blockIdx.x < S);
        float2 bias = make_float2(0.f, 0.f), scale = bias;
        if (RAW) bias = load_state(p.bias, c, p.D), scale = load_state(p.scale, c, p.D);
        if (S > 1) exchange_init(s_x);

        const int window = S * kTile, steps = (p.T + window - 1) / window;
        Seen seen;
        float carry = 0.f;  // threads 0 to 63: c of a channel behind the window
        for (int turn = 0; turn < steps; ++turn) {
            const int step = steps - 1 - turn;
            const int tile = step * window + rank * kTile, t = tile + warp * kTokens;
            const Tokens tok = look_up(p, t, kTokens, lane, seen);
            Raw raw;
            load(q, t, c, tok.own, raw);

            float2 a[kTokens], u[kTokens];
            float2 A = splat(1.f), H = splat(0.f);
#pragma unroll
            for (int k = 0; k < kTokens; ++k) {
                a[k] = splat(1.f), u[k] = splat(0.f);
                if (tok.own >> k & 1u) {
                    const float2 z = unpack<TG>(raw.z[k]), y = BETA ? unpack<TG>(raw.y[k]) : z;
                    token_map<RAW, BETA, MODE>(unpack<TA>(raw.x[k]), z, y, bias, scale, p.sigmoid, a[k], u[k]);
                }
                if (tok.first >> k & 1u) {
                    H = fma2(a[k], first_state(p, tok, k, c), u[k]);
                } else {
                    H = fma2(a[k], H, u[k]);
                    A = A * a[k];
                }
            }
            float2 rev = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = kTokens - 1; k >= 0; --k) {
                float2 d = unpack<TA>(raw.d[k]);
                if (tok.last >> k & 1u) add_final(q, tok, k, c, d);
                rev = a[k] * (d + rev);
                if (tok.first >> k & 1u) rev = splat(0.f);
            }
            if (tok.first) A = splat(kBegins);
            *reinterpret_cast<float4 *>(&s_fwd[warp][2 * lane]) = make_float4(A.x, H.x, A.y, H.y);
            *reinterpret_cast<float4 *>(&s_rev.map[warp][2 * lane]) = make_float4(A.x, rev.x, A.y, rev.y);
            __syncthreads();
            if (threadIdx.x < 64) {
                meet<true>(s_rev, s_x, S, rank, turn, threadIdx.x, carry, p.err);
            } else if (threadIdx.x < 128) {  // the states before the runs, in their place
                const int k = threadIdx.x - 64, ch = (int)(blockIdx.x / S) * 64 + k;
                float v = tile < p.T && ch < p.D ? p.chunk[(size_t)(tile / kChunk) * p.D + ch] : 0.f;
                for (int w = 0; w < kWarps; ++w) {
                    const float2 r = s_fwd[w][k];
                    s_fwd[w][k].x = v;
                    v = apply(r, v);
                }
            }
            __syncthreads();
            float2 dc = *reinterpret_cast<const float2 *>(&s_rev.h[warp][2 * lane]);
            const float4 hh = *reinterpret_cast<const float4 *>(&s_fwd[warp][2 * lane]);
            float2 h = make_float2(hh.x, hh.z);

            float2 prev[kTokens];
#pragma unroll
            for (int k = 0; k < kTokens; ++k) {
                if (tok.first >> k & 1u) h = first_state(p, tok, k, c);
                prev[k] = h;
                h = fma2(a[k], h, u[k]);
            }
            TA *dx = static_cast<TA *>(q.dx) + (int64_t)t * q.dxs + c;
            TG *dg = static_cast<TG *>(q.dg) + (int64_t)t * q.dgs + c;
            TG *db = BETA ? static_cast<TG *>(q.db) + (int64_t)t * q.dbs + c : nullptr;
#pragma unroll
            for (int k = kTokens - 1; k >= 0; --k) {
                if (!(tok.own >> k & 1u)) continue;  // hands c on
                float2 dh = unpack<TA>(raw.d[k]);
                if (tok.last >> k & 1u) add_final(q, tok, k, c, dh);
                dh = dh + dc;
                const float2 z = unpack<TG>(raw.z[k]), y = BETA ? unpack<TG>(raw.y[k]) : z;
                const float2 x = unpack<TA>(raw.x[k]);
                const Terms g = gate_terms<RAW, BETA, MODE>(z, y, bias, scale, p.sigmoid);
                dc = a[k] * dh;
                float2 d = dc * prev[k];
                if (MODE != kNone) d = fma2(g.dn * g.i * x, dh, d);
                if (RAW) {
                    sums.scale = fma2(d, g.soft, sums.scale);
                    d = d * g.dgdz;
                    sums.bias = sums.bias + d;
                }
                if (ok0) {
                    const float2 w = g.n * dh;
                    store_pair<TA>(dx + k * q.dxs, w * g.i, p.vec, ok1);
                    store_pair<TG>(dg + k * q.dgs, d, p.vec, ok1);
                    if (BETA) store_pair<TG>(db + k * q.dbs, w * x * g.di, p.vec, ok1);
                }
                if (tok.first >> k & 1u) {
                    const int row = __shfl_sync(0xffffffffu, tok.row, k);
                    if (q.dinit) store_state(q.dinit + (size_t)row * p.D, c, p.D, dc);
                    dc = splat(0.f);
                }
            }
        }
        if (RAW) {  // sums over the block's warps, then over the cluster's blocks
            const int par = steps & 1;  // one turn more of the exchange
            float4 *mine = reinterpret_cast<float4 *>(&s_fwd[warp][2 * lane]);
            __syncthreads();
            *mine = make_float4(sums.bias.x, sums.scale.x, sums.bias.y, sums.scale.y);
            __syncthreads();
            if (threadIdx.x < 64) {
                const int k = threadIdx.x, ch = (int)(blockIdx.x / S) * 64 + k;
                float2 v = s_fwd[0][k];
                for (int w = 1; w < kWarps; ++w) v = v + s_fwd[w][k];
                if (S > 1) {
                    if (k == 0) exchange_expect(s_x, par, S);
                    for (int r = 0; r < S; ++r) exchange_send(s_x, par, rank, r, k, v);
                    exchange_wait(s_x, par, steps >> 1, p.err);
                    v = s_x.map[par][0][k];
                    for (int r = 1; r < S; ++r) v = v + s_x.map[par][r][k];
                }
                if (rank == 0 && ch < p.D) {
                    if (q.dbias) q.dbias[ch] = v.x;
                    if (q.dscale) q.dscale[ch] = v.y;
                }
            }
        }
        if (S > 1) {  // no block leaves while another may still send to it
            cluster_arrive();
            cluster_wait();
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
    const int cb = (q.f.D + 63) / 64, tile = Backward<TA, TG, RAW, BETA>::kTile;
    int S = 1;
    const cudaError_t e = cluster_blocks((const void *)kernel, 0, cb, (q.f.T + tile - 1) / tile, &S);
    if (e != cudaSuccess) return e;
    return launch_clusters(cb, S, 0, stream, kernel, q);
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
