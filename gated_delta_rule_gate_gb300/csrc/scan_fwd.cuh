// scan_fwd.cuh -- gdn_scan: the gated linear recurrence, parallel over channels
// and along time, in one launch.
//
// h_t = a_t h_{t-1} + u_t is a composition of affine maps: a run of tokens takes
// h to A h + H with A the product of its a and H its result from a zero state.
// A warp takes kTokens tokens of 64 channels (a lane two of them), a block the
// runs of its warps, a cluster of S blocks the tiles of its blocks; the cluster
// walks the whole token axis of its channels in windows of S tiles and carries
// the state from window to window in registers.  Per window: every warp folds
// its run to (A, H); the block's warps exchange theirs in shared memory, the
// blocks theirs in distributed shared memory (one cluster barrier); every warp
// then has the state before its run, in the same order of operations on every
// run, and walks its tokens, which have stayed in registers, a second time to
// write o.  The loads of the next window are in flight meanwhile, so x, decay and
// beta cross HBM once.  A request's first token takes in the request's initial
// state and nothing of the token before it, so that ragged requests need nothing else.
#pragma once

#include "scan_cluster.cuh"

namespace gdn {
namespace scan {

// Empty requests keep their state; bad slot ids and decreasing offsets are
// reported.  Once per channel block, the requests shared out over the warps.
__device__ __forceinline__ void request_duties(const Args &p, int warps, int warp, int lane, int c, bool report) {
    for (int b = warp; b < p.B; b += warps) {
        int t0, t1;
        request_tokens(p, b, t0, t1);
        const int row = request_row(p, b);
        if (report && lane == 0 && p.err) {
            if (row < 0) atomicOr(p.err, kErrBadSlot);
            if (p.cu && clamped_offset(p, b + 1) < clamped_offset(p, b)) atomicOr(p.err, kErrOverlap);
        }
        if (t0 == t1 && row >= 0 && p.fin && p.fin != p.init) {
            const size_t at = (size_t)row * p.D;
            store_state(p.fin + at, c, p.D, p.init ? load_state(p.init + at, c, p.D) : make_float2(0.f, 0.f));
        }
    }
}

template <typename TA, typename TG, bool RAW, bool BETA>
struct Forward {
    static constexpr int kTokens = sizeof(TA) == 2 && sizeof(TG) == 2 ? 16 : 8;
    static constexpr int kTile = kWarps * kTokens;

    struct Raw {
        pair_t<TA> x[kTokens];
        pair_t<TG> z[kTokens], y[BETA ? kTokens : 1];
    };

    static __device__ __forceinline__ void load(const Args &p, int t, int c, unsigned own, Raw &r) {
        const TA *x = static_cast<const TA *>(p.x) + (int64_t)t * p.xs + c;
        const TG *z = static_cast<const TG *>(p.decay) + (int64_t)t * p.gs + c;
        const TG *y = BETA ? static_cast<const TG *>(p.beta) + (int64_t)t * p.bs + c : nullptr;
        const bool vec = p.vec, ok1 = c + 1 < p.D;
        if (c >= p.D) own = 0u;
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            const bool on = own >> k & 1u;
            r.x[k] = on ? load_pair<TA>(x + k * p.xs, vec, ok1) : zero_pair<TA>();
            r.z[k] = on ? load_pair<TG>(z + k * p.gs, vec, ok1) : zero_pair<TG>();
            if (BETA) r.y[k] = on ? load_pair<TG>(y + k * p.bs, vec, ok1) : zero_pair<TG>();
        }
    }

    template <int MODE>
    static __device__ __forceinline__ void gates(const Args &p, const Raw &r, float2 bias, float2 scale, float2 *a,
                                                 float2 *u) {
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            const float2 z = unpack<TG>(r.z[k]);
            const float g0 = log_decay<RAW>(z.x, bias.x, scale.x), g1 = log_decay<RAW>(z.y, bias.y, scale.y);
            a[k] = make_float2(expf(g0), expf(g1));
            u[k] = unpack<TA>(r.x[k]);
            if (BETA) {
                float2 y = unpack<TG>(r.y[k]);
                if (p.sigmoid) y = make_float2(sigmoid(y.x), sigmoid(y.y));
                u[k].x *= y.x;
                u[k].y *= y.y;
            }
            if (MODE != kNone) {
                u[k].x *= input_scale<MODE>(g0, a[k].x);
                u[k].y *= input_scale<MODE>(g1, a[k].y);
            }
        }
    }

    static __device__ __forceinline__ void run(const Args &p) {
        __shared__ float4 s_warp[2][kWarps][32];
        __shared__ float4 s_rank[2][kMaxCluster][32];
        const int S = cluster_size(), rank = cluster_rank();
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int c = (int)(blockIdx.x / S) * 64 + 2 * lane;
        const bool ok0 = c < p.D, ok1 = c + 1 < p.D;
        if (S > 1) cluster_arrive();  // waited for before the first remote store

        const int window = S * kTile, steps = (p.T + window - 1) / window;
        int t = rank * kTile + warp * kTokens;
        Seen seen;
        Tokens tok = look_up(p, t, kTokens, lane, seen);
        Raw raw;
        load(p, t, c, tok.own, raw);
        float2 bias = make_float2(0.f, 0.f), scale = bias;
        if (RAW) bias = load_state(p.bias, c, p.D), scale = load_state(p.scale, c, p.D);
        request_duties(p, S * kWarps, rank * kWarps + warp, lane, c, blockIdx.x < S);
        if (S > 1) cluster_wait();

        float2 carry = make_float2(0.f, 0.f);  // the state before the window
        for (int step = 0; step < steps; ++step) {
            const int par = step & 1;
            float2 a[kTokens], u[kTokens];
            if (p.mode == kNone) gates<kNone>(p, raw, bias, scale, a, u);
            else if (p.mode == kLerp) gates<kLerp>(p, raw, bias, scale, a, u);
            else gates<kUnit>(p, raw, bias, scale, a, u);
            const Tokens now = tok;
            const int tn = t;
            // tokens of no request hand the state on; a first token takes its request's initial state
            float4 run = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
            for (int k = 0; k < kTokens; ++k) {
                if (!(now.own >> k & 1u)) a[k] = make_float2(1.f, 1.f), u[k] = make_float2(0.f, 0.f);
                if (now.first >> k & 1u) {
                    const int row = __shfl_sync(0xffffffffu, now.row, k);
                    if (p.init) {
                        const float2 h0 = load_state(p.init + (size_t)row * p.D, c, p.D);
                        u[k].x = fmaf(a[k].x, h0.x, u[k].x);
                        u[k].y = fmaf(a[k].y, h0.y, u[k].y);
                    }
                    run = make_float4(kBegins, u[k].x, kBegins, u[k].y);
                } else {
                    run.y = fmaf(a[k].x, run.y, u[k].x);
                    run.w = fmaf(a[k].y, run.w, u[k].y);
                    run.x *= a[k].x;
                    run.z *= a[k].y;
                }
            }
            if (now.first) run.x = run.z = kBegins;
            t += window;
            if (step + 1 < steps) {
                tok = look_up(p, t, kTokens, lane, seen);
                load(p, t, c, tok.own, raw);
            }
            s_warp[par][warp][lane] = run;
            __syncthreads();
            float4 before = make_float4(1.f, 0.f, 1.f, 0.f), tile = before;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) before = tile;
                fold(tile, s_warp[par][w][lane]);
            }
            float2 h = carry;
            if (S > 1) {
                for (int r = warp; r < S; r += kWarps) store_remote(&s_rank[par][rank][lane], r, tile);
                cluster_arrive();
                cluster_wait();
                for (int r = 0; r < S; ++r) {
                    if (r == rank) h = carry;
                    carry = apply(s_rank[par][r][lane], carry);
                }
            } else {
                carry = apply(tile, carry);
            }
            h = apply(before, h);
            if (p.chunk && tn % kChunk == 0 && tn < p.T)
                store_state(p.chunk + (size_t)(tn / kChunk) * p.D, c, p.D, h);
            TA *o = static_cast<TA *>(p.o) + (int64_t)tn * p.os + c;
#pragma unroll
            for (int k = 0; k < kTokens; ++k) {
                if (now.first >> k & 1u) h = u[k];
                else h = make_float2(fmaf(a[k].x, h.x, u[k].x), fmaf(a[k].y, h.y, u[k].y));
                if ((now.own >> k & 1u) && ok0) store_pair<TA>(o + k * p.os, h, p.vec, ok1);
                if ((now.last >> k & 1u) && p.fin) {
                    const int row = __shfl_sync(0xffffffffu, now.row, k);
                    store_state(p.fin + (size_t)row * p.D, c, p.D, h);
                }
            }
        }
    }
};

template <typename TA, typename TG, bool RAW, bool BETA>
__global__ void __launch_bounds__(kWarps * 32, 2) scan_kernel(const __grid_constant__ Args p) {
    Forward<TA, TG, RAW, BETA>::run(p);
}

template <typename TA, typename TG, bool RAW, bool BETA>
cudaError_t launch_one(const Args &p, cudaStream_t stream) {
    auto kernel = scan_kernel<TA, TG, RAW, BETA>;
    int per_sm = 1;
    cudaError_t e = blocks_per_sm((const void *)kernel, kWarps * 32, 0, &per_sm);
    if (e == cudaSuccess) e = large_clusters((const void *)kernel);
    if (e != cudaSuccess) return e;
    const int cb = (p.D + 63) / 64, tile = Forward<TA, TG, RAW, BETA>::kTile;
    const int S = cluster_blocks(cb, (p.T + tile - 1) / tile, per_sm * sm_count());
    return launch_clusters(kernel, p, cb, S, stream);
}

template <typename TA, typename TG>
cudaError_t launch_types(const Args &p, cudaStream_t stream) {
    if (p.bias) return p.beta ? launch_one<TA, TG, true, true>(p, stream) : launch_one<TA, TG, true, false>(p, stream);
    return p.beta ? launch_one<TA, TG, false, true>(p, stream) : launch_one<TA, TG, false, false>(p, stream);
}

}  // namespace scan
}  // namespace gdn
