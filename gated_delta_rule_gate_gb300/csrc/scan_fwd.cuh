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
// blocks theirs in distributed shared memory; every warp
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

template <typename TA, typename TG, bool RAW, bool BETA, int MODE>
struct Forward {
    static constexpr int kTokens = sizeof(TA) == 2 ? 16 : 8;
    static constexpr int kTile = kWarps * kTokens;

    struct Input {
        Stage<TA, kTokens> x;
        Stage<TG, kTokens> z, y[BETA ? 1 : 0];
    };
    struct Shared {
        Exchange x;
        float4 map[2][kWarps][32];
        Input in[kWarps];
    };

    static __device__ __forceinline__ void fill(const Args &p, Input &in, int t, int block, unsigned own, int lane) {
        in.x.fill(p.x, p.xs, t, block, own, p.D, p.wide, p.vec, lane);
        in.z.fill(p.decay, p.gs, t, block, own, p.D, p.wide, p.vec, lane);
        if constexpr (BETA) in.y[0].fill(p.beta, p.bs, t, block, own, p.D, p.wide, p.vec, lane);
    }

    // a, u of the warp's tokens and its map.  PLAIN: all of them inside one request.
    template <bool PLAIN>
    static __device__ __forceinline__ float4 first_walk(const Args &p, const Input &in, const Tokens &tok, int c,
                                                        int lane, float2 bias, float2 scale, float2 (&a)[kTokens],
                                                        float2 (&u)[kTokens]) {
        float2 A = splat(1.f), H = splat(0.f);
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            float2 y = splat(0.f);
            if constexpr (BETA) y = in.y[0].at(k, lane);
            token_map<RAW, BETA, MODE>(in.x.at(k, lane), in.z.at(k, lane), y, bias, scale, p.sigmoid, a[k], u[k]);
            if (!PLAIN) {  // tokens of no request hand the state on
                if (!(tok.own >> k & 1u)) a[k] = splat(1.f), u[k] = splat(0.f);
                if (tok.first >> k & 1u) {  // takes in the request's initial state
                    const int row = __shfl_sync(0xffffffffu, tok.row, k);
                    if (p.init) u[k] = fma2(a[k], load_state(p.init + (size_t)row * p.D, c, p.D), u[k]);
                    H = splat(0.f);
                }
            }
            H = !PLAIN && (tok.first >> k & 1u) ? u[k] : fma2(a[k], H, u[k]);
            A = A * a[k];
        }
        if (!PLAIN && tok.first) A = splat(kBegins);
        return map_of(A, H);
    }

    template <bool PLAIN>
    static __device__ __forceinline__ void second_walk(const Args &p, const Tokens &tok, int t, int c,
                                                       const float2 (&a)[kTokens], const float2 (&u)[kTokens],
                                                       float2 h) {
        TA *o = static_cast<TA *>(p.o) + (int64_t)t * p.os + c;
        const bool ok0 = c < p.D, ok1 = c + 1 < p.D;
        if (PLAIN && p.vec) {
#pragma unroll
            for (int k = 0; k < kTokens; ++k) {
                h = fma2(a[k], h, u[k]);
                if (ok0) *reinterpret_cast<pair_t<TA> *>(o + k * p.os) = pack<TA>(h);
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            h = tok.first >> k & 1u ? u[k] : fma2(a[k], h, u[k]);
            if ((tok.own >> k & 1u) && ok0) store_pair<TA>(o + k * p.os, h, p.vec, ok1);
            if ((tok.last >> k & 1u) && p.fin) {
                const int row = __shfl_sync(0xffffffffu, tok.row, k);
                store_state(p.fin + (size_t)row * p.D, c, p.D, h);
            }
        }
    }

    static __device__ __forceinline__ void run(const Args &p, Shared &s) {
        const int S = cluster_size(), rank = cluster_rank();
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int block = (int)(blockIdx.x / S), c = block * 64 + 2 * lane;
        constexpr unsigned kAll = (1u << kTokens) - 1u;

        const int window = S * kTile, steps = (p.T + window - 1) / window;
        int t = rank * kTile + warp * kTokens;
        Seen seen;
        Input &in = s.in[warp];
        Tokens tok = look_up(p, t, kTokens, lane, seen);
        fill(p, in, t, block, tok.own, lane);
        float2 bias = splat(0.f), scale = bias;
        if (RAW) bias = load_state(p.bias, c, p.D), scale = load_state(p.scale, c, p.D);
        request_duties(p, S * kWarps, rank * kWarps + warp, lane, c, blockIdx.x < S);
        if (S > 1) exchange_init(s.x);

        float2 carry = splat(0.f);  // the state before the window
        for (int step = 0; step < steps; ++step) {
            const int par = step & 1;
            float2 a[kTokens], u[kTokens];
            const Tokens now = tok;
            const int tn = t;
            const bool plain = now.own == kAll && !(now.first | now.last);
            stage_wait();
            s.map[par][warp][lane] = plain ? first_walk<true>(p, in, now, c, lane, bias, scale, a, u)
                                           : first_walk<false>(p, in, now, c, lane, bias, scale, a, u);
            t += window;
            __syncwarp();
            if (step + 1 < steps) {
                tok = look_up(p, t, kTokens, lane, seen);
                fill(p, in, t, block, tok.own, lane);
            }
            // the runs of the block's warps: those before this warp's, and all
            const bool resets = __syncthreads_or(now.first);
            float2 A = splat(1.f), H = splat(0.f), beforeA = A, beforeH = H;
            if (!resets) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    if (w == warp) beforeA = A, beforeH = H;
                    fold<false>(A, H, s.map[par][w][lane]);
                }
            } else {
                for (int w = 0; w < kWarps; ++w) {
                    if (w == warp) beforeA = A, beforeH = H;
                    fold<true>(A, H, s.map[par][w][lane]);
                }
            }
            float2 h = carry;
            if (S > 1) {
                if (threadIdx.x == 0) exchange_expect(s.x, par, S);
                for (int r = warp; r < S; r += kWarps) exchange_send(s.x, par, rank, r, lane, map_of(A, H));
                exchange_wait(s.x, par, step >> 1, p.err);
                for (int r = 0; r < rank; ++r) carry = apply(s.x.map[par][r][lane], carry);
                h = carry;
                for (int r = rank; r < S; ++r) carry = apply(s.x.map[par][r][lane], carry);
            } else {
                carry = apply(map_of(A, H), carry);
            }
            h = apply(map_of(beforeA, beforeH), h);
            if (p.chunk && tn % kChunk == 0 && tn < p.T)
                store_state(p.chunk + (size_t)(tn / kChunk) * p.D, c, p.D, h);
            if (plain) second_walk<true>(p, now, tn, c, a, u, h);
            else second_walk<false>(p, now, tn, c, a, u, h);
        }
        if (S > 1) {  // no block leaves while another may still send to it
            cluster_arrive();
            cluster_wait();
        }
    }
};

template <typename TA, typename TG, bool RAW, bool BETA, int MODE>
__global__ void __launch_bounds__(kWarps * 32, 2) scan_kernel(const __grid_constant__ Args p) {
    using F = Forward<TA, TG, RAW, BETA, MODE>;
    extern __shared__ __align__(16) unsigned char smem[];
    F::run(p, *reinterpret_cast<typename F::Shared *>(smem));
}

template <typename TA, typename TG, bool RAW, bool BETA, int MODE>
cudaError_t launch_one(const Args &p, cudaStream_t stream) {
    using F = Forward<TA, TG, RAW, BETA, MODE>;
    auto kernel = scan_kernel<TA, TG, RAW, BETA, MODE>;
    const int cb = (p.D + 63) / 64;
    int S = 1;
    const cudaError_t e =
        cluster_blocks((const void *)kernel, sizeof(typename F::Shared), cb, (p.T + F::kTile - 1) / F::kTile, &S);
    if (e != cudaSuccess) return e;
    return launch_clusters(kernel, p, cb, S, sizeof(typename F::Shared), stream);
}

template <typename TA, typename TG, bool RAW, bool BETA>
cudaError_t launch_mode(const Args &p, cudaStream_t stream) {
    if (p.mode == kNone) return launch_one<TA, TG, RAW, BETA, kNone>(p, stream);
    if (p.mode == kLerp) return launch_one<TA, TG, RAW, BETA, kLerp>(p, stream);
    return launch_one<TA, TG, RAW, BETA, kUnit>(p, stream);
}

template <typename TA, typename TG>
cudaError_t launch_types(const Args &p, cudaStream_t stream) {
    if (p.bias)
        return p.beta ? launch_mode<TA, TG, true, true>(p, stream) : launch_mode<TA, TG, true, false>(p, stream);
    return p.beta ? launch_mode<TA, TG, false, true>(p, stream) : launch_mode<TA, TG, false, false>(p, stream);
}

}  // namespace scan
}  // namespace gdn
