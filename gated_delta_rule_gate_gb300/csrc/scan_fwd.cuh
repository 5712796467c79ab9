// scan_fwd.cuh -- gdn_scan: the gated linear recurrence, parallel over channels
// and along time, in one launch.
//
// h_t = a_t h_{t-1} + u_t is a composition of affine maps: a run of tokens takes
// h to A h + H with A the product of its a (kept as its root, see scan_cluster.cuh) and
// H its result from a zero state.
// A warp takes kTokens tokens of 64 channels (a lane two of them), a block the
// runs of its warps, a cluster of S blocks the tiles of its blocks; the cluster
// walks the whole token axis of its channels in windows of S tiles and carries
// the state from window to window in registers.  Per window: every warp folds
// its run to its map; the block's warps exchange theirs in shared memory, the
// blocks theirs in distributed shared memory (Meet); every warp
// then has the state before its run, in the same order of operations on every
// run, and walks its tokens, which have stayed in registers, a second time to
// write o.  The loads of the next window are in flight meanwhile, so x, decay and
// beta cross HBM once.  A request's first token takes in the request's initial
// state and nothing of the token before it, so that ragged requests need nothing else.
//
// 8 ragged requests of 16384 tokens together x 4096 channels fp16 with raw gates, input
// gate and states take 163 us, where HBM alone would take 79.  Half of it is the issue of
// instructions, of which the gates' functions are the most (88 a token and 64 channels, 52 %
// of the slots), the other half each window's wait for its loads and for the exchange, with
// 3 warps a scheduler to fill it.  With the decay given as its logarithm and no input gate
// 32768 x 2048 bf16 takes 85 us, 70 % of HBM.
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

struct Maps {
    CUtensorMap x, z, y, o;
};

template <int WARPS, bool WIDE, typename TA, typename TG, bool RAW, bool BETA, int MODE>
struct Forward {
    // Long runs cost less of the exchange; with fp32 tensors they would leave room for
    // one block an SM (32768 tokens x 2048 bf16 with fp32 gates: 169 us at 8, 190 at 16; with
    // bf16 gates 16 are the faster).
    static constexpr int kTokens = sizeof(TA) == 2 && sizeof(TG) == 2 ? 16 : 8;
    static constexpr int kTile = WARPS * kTokens;
    static_assert(kTile * kMaxCluster <= kMaxWindow, "token counts are checked against the largest window");

    struct Input {
        Stage<TA, kTokens> x;
        Stage<TG, kTokens> z, y[BETA ? 1 : 0];
    };
    struct alignas(128) Shared {
        Input in[WARPS];
        Stage<TA, kTokens> out[WARPS];
        Exchange x;
        Meeting<WARPS> meet;
        uint64_t bar[WARPS];
    };

    // The warp's tokens t, ... to its stage, by the asynchronous copies of WIDE rows on
    // their way there; otherwise the tokens of the window after on their way to L2.
    static __device__ __forceinline__ void fill(const Args &p, const Maps &m, Input &in, uint64_t *bar, int t, int window,
                                                int block, unsigned own, int lane) {
        if (WIDE) {
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(bar, sizeof(Input));
                in.x.fill(m.x, t, block, bar);
                in.z.fill(m.z, t, block, bar);
                if constexpr (BETA) in.y[0].fill(m.y, t, block, bar);
            }
            return;
        }
        in.x.prefetch_row(p.x, p.xs, t + window, p.T, block, p.D, lane);
        in.z.prefetch_row(p.decay, p.gs, t + window, p.T, block, p.D, lane);
        if constexpr (BETA) in.z.prefetch_row(p.beta, p.bs, t + window, p.T, block, p.D, lane);
        if (inside(p, t, kTokens, block)) {
            in.x.fill_words(p.x, p.xs, t, block, own, p.D, lane);
            in.z.fill_words(p.decay, p.gs, t, block, own, p.D, lane);
            if constexpr (BETA) in.y[0].fill_words(p.beta, p.bs, t, block, own, p.D, lane);
        } else {
            in.x.fill_each(p.x, p.xs, t, block, own, p.D, lane);
            in.z.fill_each(p.decay, p.gs, t, block, own, p.D, lane);
            if constexpr (BETA) in.y[0].fill_each(p.beta, p.bs, t, block, own, p.D, lane);
        }
    }

    // a, u of the warp's tokens and its map.  PLAIN: all of them inside one request, and their
    // channels whole words where they are stored as such.
    template <bool PLAIN>
    static __device__ __forceinline__ float4 first_walk(const Args &p, const Input &in, const Tokens &tok, int c,
                                                        int lane, float2 bias, float2 scale, float2 (&a)[kTokens],
                                                        float2 (&u)[kTokens]) {
        float2 sum = splat(0.f), H = splat(0.f);
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            float2 y = splat(0.f);
            if constexpr (BETA) y = in.y[0].at(k, lane);
            const Gates g = token_gates<RAW, BETA, MODE>(in.z.at(k, lane), y, bias, scale, p.sigmoid);
            float2 own_g = g.g;
            a[k] = g.a;
            u[k] = scaled<BETA, MODE>(in.x.at(k, lane), g.n, g.i);
            if (!PLAIN) {  // tokens of no request hand the state on
                if (!(tok.own >> k & 1u)) a[k] = splat(1.f), own_g = u[k] = splat(0.f);
                if (tok.first >> k & 1u) {  // takes in the request's initial state
                    const int row = __shfl_sync(0xffffffffu, tok.row, k);
                    if (p.init) u[k] = fma2(a[k], load_state(p.init + (size_t)row * p.D, c, p.D), u[k]);
                    H = splat(0.f);
                }
            }
            H = !PLAIN && (tok.first >> k & 1u) ? u[k] : fma2(a[k], H, u[k]);
            sum = sum + own_g;
        }
        const float2 R = !PLAIN && tok.first ? splat(kBegins) : root_of(sum);
        return make_float4(R.x, H.x, R.y, H.y);
    }

    // o of the warp's tokens, which a plain run of whole words hands to an asynchronous copy.
    template <bool PLAIN>
    static __device__ __forceinline__ void second_walk(const Args &p, const Maps &m, Stage<TA, kTokens> &out,
                                                       const Tokens &tok, int t, int block, int lane,
                                                       const float2 (&a)[kTokens], const float2 (&u)[kTokens],
                                                       float2 h) {
        const int c = block * 64 + 2 * lane;
        if (PLAIN && WIDE) {
            if (lane == 0) ptx::bulk_wait_read();  // the last copy has left the stage
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kTokens; ++k) {
                h = fma2(a[k], h, u[k]);
                out.v[k][lane] = pack<TA>(h);
            }
            ptx::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                ptx::tma_store_2d(&m.o, c, t, out.v);
                ptx::bulk_commit();
            }
            return;
        }
        TA *o = static_cast<TA *>(p.o) + (int64_t)t * p.os + block * 64;
        const int n = p.D - block * 64;
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            h = !PLAIN && (tok.first >> k & 1u) ? u[k] : fma2(a[k], h, u[k]);
            if (PLAIN || (tok.own >> k & 1u)) store_row<TA>(o + k * p.os, h, lane, n);
            if (!PLAIN && (tok.last >> k & 1u) && p.fin) {
                const int row = __shfl_sync(0xffffffffu, tok.row, k);
                store_state(p.fin + (size_t)row * p.D, c, p.D, h);
            }
        }
    }

    static __device__ __forceinline__ void run(const Args &p, const Maps &m, Shared &s) {
        const Place at = place_of(p);
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int block = (int)(blockIdx.x / at.size), c = block * 64 + 2 * lane;
        constexpr unsigned kAll = (1u << kTokens) - 1u;

        const int window = at.S * kTile, steps = windows(at, window);
        int t = at.base + at.rank * kTile + warp * kTokens;
        Input &in = s.in[warp];
        uint64_t *bar = &s.bar[warp];
        if (lane == 0) {
            ptx::mbar_init(bar, 1);
            ptx::fence_mbar_init();
        }
        __syncwarp();
        ptx::grid_wait();
        Seen seen;
        Tokens tok = look_up(p, at.lo, at.hi, t, kTokens, lane, seen);
        if (steps > 0) fill(p, m, in, bar, t, window, block, tok.own, lane);
        float2 bias = splat(0.f), scale = bias;
        if (RAW) bias = load_state(p.bias, c, p.D), scale = load_state(p.scale, c, p.D);
        if (at.size > 1) exchange_init(s.x);
        request_duties(p, at.size * WARPS, at.me * WARPS + warp, lane, c, blockIdx.x < at.size);

        const bool whole = !WIDE || whole_words<TA>(p.D, block);
        float carry = 0.f;  // the state of this thread's channel (see Meet) before the window
        for (int step = 0; step < steps; ++step, t += window) {
            const int par = step & 1;
            float2 a[kTokens], u[kTokens];
            const Tokens now = tok;
            const bool plain = now.own == kAll && !(now.first | now.last) && whole;
            if (WIDE) {
                if (!ptx::mbar_wait(bar, par) && p.err) atomicOr(p.err, kErrTimeout);
            } else {
                __syncwarp();
            }
            *reinterpret_cast<float4 *>(&s.meet.map[warp][2 * lane]) =
                plain ? first_walk<true>(p, in, now, c, lane, bias, scale, a, u)
                      : first_walk<false>(p, in, now, c, lane, bias, scale, a, u);
            __syncthreads();
            Meet<false, WARPS> meet;
            const float2 tile = meet.send(s.meet, s.x, at, step);
            if (step + 1 < steps) {  // while the maps are on their way
                tok = look_up(p, at.lo, at.hi, t + window, kTokens, lane, seen);
                if (WIDE) fill(p, m, in, bar, t + window, window, block, tok.own, lane);
            }
            meet.receive(s.meet, s.x, at, step, tile, carry, p.err);
            __syncthreads();
            const float2 h = *reinterpret_cast<const float2 *>(&s.meet.h[warp][2 * lane]);
            if (p.chunk && t % kChunk == 0 && t >= at.lo && t < at.hi)
                store_state(p.chunk + (size_t)(t / kChunk) * p.D, c, p.D, h);
            if (plain) second_walk<true>(p, m, s.out[warp], now, t, block, lane, a, u, h);
            else second_walk<false>(p, m, s.out[warp], now, t, block, lane, a, u, h);
            // through registers, which a and u have left
            if (!WIDE && step + 1 < steps) fill(p, m, in, bar, t + window, window, block, tok.own, lane);
        }
        if (lane == 0) ptx::bulk_wait();
        if (at.size > 1) {  // no block leaves while another may still send to it
            cluster_arrive();
            cluster_wait();
        }
    }
};

// 16 warps an SM.
template <int WARPS, bool WIDE, typename TA, typename TG, bool RAW, bool BETA, int MODE>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) scan_kernel(const __grid_constant__ Args p,
                                                                     const __grid_constant__ Maps m) {
    using F = Forward<WARPS, WIDE, TA, TG, RAW, BETA, MODE>;
    extern __shared__ __align__(128) unsigned char smem[];
    F::run(p, m, *reinterpret_cast<typename F::Shared *>(smem));
}

template <int WARPS, bool WIDE, typename TA, typename TG, bool RAW, bool BETA, int MODE>
cudaError_t blocks_for(const Args &p, int *S) {
    using F = Forward<WARPS, WIDE, TA, TG, RAW, BETA, MODE>;
    return cluster_blocks((const void *)scan_kernel<WARPS, WIDE, TA, TG, RAW, BETA, MODE>, WARPS,
                          sizeof(typename F::Shared), (p.D + 63) / 64, (p.T + F::kTile - 1) / F::kTile, S);
}
template <int WARPS, bool WIDE, typename TA, typename TG, bool RAW, bool BETA, int MODE>
cudaError_t launch_blocks(const Args &p, int S, cudaStream_t stream) {
    using F = Forward<WARPS, WIDE, TA, TG, RAW, BETA, MODE>;
    Maps m = {};
    Args q = p;
    share_out(q, S, F::kTile);
    if (WIDE && !(make_token_map(&m.x, p.x, type_of<TA>(), p.xs, p.D, p.T, F::kTokens) &&
                  make_token_map(&m.z, p.decay, type_of<TG>(), p.gs, p.D, p.T, F::kTokens) &&
                  (!BETA || make_token_map(&m.y, p.beta, type_of<TG>(), p.bs, p.D, p.T, F::kTokens)) &&
                  make_token_map(&m.o, p.o, type_of<TA>(), p.os, p.D, p.T, F::kTokens)))
        return cudaErrorInvalidValue;
    // A pass that keeps states is one of training, between gradients that fill the SMs'
    // shared memory: set up while one still runs, its blocks take the places that come
    // free first, and the whole grid is slower than one set up afterwards (a training
    // pass of 4096 x 2048 bf16 105 us, 97 so; 32768 x 2048 472 and 466), but for one
    // window or two, where the launch counts (999 x 1000 fp32 33.1 us, 34.4 not early).
    // Without states always early (4096 x 1024 23.0 us, 24.7 not).
    const int64_t window = (int64_t)(S / q.groups) * F::kTile;
    const bool early = !p.chunk || p.T <= 2 * q.groups * window;
    return launch_clusters((p.D + 63) / 64, S, WARPS, sizeof(typename F::Shared), early, stream,
                           scan_kernel<WARPS, WIDE, TA, TG, RAW, BETA, MODE>, q, m);
}

// Of 16-bit tensors blocks of 4 warps are shared out more evenly and wait for fewer
// others, but a cluster has 16 at most: blocks of 8 where it gets more warps from
// them.  us with 4 and 8, bf16, raw gates: 16384 x 4096 ragged 163 and 165, 16384 x 2560
// 102 and 112, 32768 x 2048 142 and 143, 32768 x 512 88 and 80.  Tiles of fp32 tensors are
// half as long, and rows that are read by words want more of them on their way: 8
// (16384 x 2048 fp32 104 and 103; 16384 x 2047 bf16 240 and 196).  A pass that keeps states
// takes 8 too: the small blocks leave a gradient that is set up beside them no room for
// two on an SM (a training pass of 32768 x 2048 471 us, 466 with 8).
template <bool WIDE, typename TA, typename TG, bool RAW, bool BETA, int MODE>
cudaError_t launch_one(const Args &p, cudaStream_t stream) {
    int eights = 1;
    cudaError_t e = blocks_for<8, WIDE, TA, TG, RAW, BETA, MODE>(p, &eights);
    if constexpr (WIDE && sizeof(TA) == 2 && sizeof(TG) == 2) {
        if (e == cudaSuccess && !p.chunk) {
            int fours = 1;
            e = blocks_for<4, WIDE, TA, TG, RAW, BETA, MODE>(p, &fours);
            if (e == cudaSuccess && eights * 8 <= fours * 4)
                return launch_blocks<4, WIDE, TA, TG, RAW, BETA, MODE>(p, fours, stream);
        }
    }
    return e == cudaSuccess ? launch_blocks<8, WIDE, TA, TG, RAW, BETA, MODE>(p, eights, stream) : e;
}

template <bool WIDE, typename TA, typename TG, bool RAW, bool BETA>
cudaError_t launch_mode(const Args &p, cudaStream_t stream) {
    if (p.mode == kNone) return launch_one<WIDE, TA, TG, RAW, BETA, kNone>(p, stream);
    if (p.mode == kLerp) return launch_one<WIDE, TA, TG, RAW, BETA, kLerp>(p, stream);
    return launch_one<WIDE, TA, TG, RAW, BETA, kUnit>(p, stream);
}

template <bool WIDE, typename TA, typename TG>
cudaError_t launch_types(const Args &p, cudaStream_t stream) {
    if (p.bias)
        return p.beta ? launch_mode<WIDE, TA, TG, true, true>(p, stream)
                      : launch_mode<WIDE, TA, TG, true, false>(p, stream);
    return p.beta ? launch_mode<WIDE, TA, TG, false, true>(p, stream)
                  : launch_mode<WIDE, TA, TG, false, false>(p, stream);
}

}  // namespace scan
}  // namespace gdn
