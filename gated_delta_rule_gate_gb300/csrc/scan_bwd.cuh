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
//
// 4 x 8192 x 2048 bf16 with raw and input gates 312 us, 2.9 TB/s; the pass with its forward
// 466, with the decay given as its logarithm and no input gate 249.  The issue of
// instructions (183 a token and 64 channels, 53 % of the slots) takes half of it, the waits of
// each window for its loads and the exchange the rest.  What a warp holds of its tokens
// between the walks is 64 registers of 128: with raw and input gates and an input scale 112 to
// 140 bytes a thread are spilled (64 to 164 where rows are read by words).
#pragma once

#include "scan_cluster.cuh"

namespace gdn {
namespace scan {

constexpr int kWarps = 8;

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

struct GradMaps {
    CUtensorMap x, z, y, d, dx, dz, dy;
};

template <bool WIDE, typename TA, typename TG, bool RAW, bool BETA, int MODE>
struct Backward {
    static constexpr int kTokens = 8;
    static constexpr int kTile = kWarps * kTokens;
    static_assert(kTile == kChunk, "a tile begins where the forward pass kept a state");

    // A warp's tokens; the gradients take the places of x, decay and beta.
    struct Input {
        Stage<TA, kTokens> x, d;
        Stage<TG, kTokens> z, y[BETA ? 1 : 0];
    };
    struct Rest {
        Exchange x;
        Meeting<kWarps> rev;               // (R, C) of each warp's run, and c behind it
        alignas(16) float2 fwd[kWarps][64];  // (R, H) of each warp's run; at the end its sums
        float h[kWarps][64];       // the state before it
        uint64_t bar[kWarps][2];
    };
    // Two stages where two blocks an SM have room for them, so that a window's loads
    // are on their way during the one before.
    static constexpr int kRing = 2 * kWarps * sizeof(Input) + sizeof(Rest) <= 113 * 1024 ? 2 : 1;
    struct alignas(128) Shared {
        Input in[kWarps][kRing];
        Rest r;
    };
    struct Sums {
        float2 bias, scale;
    };

    // The warp's tokens t, ... to its stage, by the asynchronous copies of WIDE rows on
    // their way there; otherwise the tokens of the window before on their way to L2.
    static __device__ __forceinline__ void fill(const GradArgs &q, const GradMaps &m, Input &in, uint64_t *bar, int t,
                                                int window, int block, unsigned own, int lane) {
        const Args &p = q.f;
        if (WIDE) {
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(bar, sizeof(Input));
                in.x.fill(m.x, t, block, bar);
                in.d.fill(m.d, t, block, bar);
                in.z.fill(m.z, t, block, bar);
                if constexpr (BETA) in.y[0].fill(m.y, t, block, bar);
            }
            return;
        }
        if (t >= window) {
            in.x.prefetch_row(p.x, p.xs, t - window, p.T, block, p.D, lane);
            in.x.prefetch_row(q.d_o, q.dos, t - window, p.T, block, p.D, lane);
            in.z.prefetch_row(p.decay, p.gs, t - window, p.T, block, p.D, lane);
            if constexpr (BETA) in.z.prefetch_row(p.beta, p.bs, t - window, p.T, block, p.D, lane);
        }
        if (inside(p, t, kTokens, block)) {
            in.x.fill_words(p.x, p.xs, t, block, own, p.D, lane);
            in.d.fill_words(q.d_o, q.dos, t, block, own, p.D, lane);
            in.z.fill_words(p.decay, p.gs, t, block, own, p.D, lane);
            if constexpr (BETA) in.y[0].fill_words(p.beta, p.bs, t, block, own, p.D, lane);
        } else {
            in.x.fill_each(p.x, p.xs, t, block, own, p.D, lane);
            in.d.fill_each(q.d_o, q.dos, t, block, own, p.D, lane);
            in.z.fill_each(p.decay, p.gs, t, block, own, p.D, lane);
            if constexpr (BETA) in.y[0].fill_each(p.beta, p.bs, t, block, own, p.D, lane);
        }
    }

    static __device__ __forceinline__ void prefetch(const GradMaps &m, int t, int block) {
        Stage<TA, kTokens>::prefetch(m.x, t, block);
        Stage<TA, kTokens>::prefetch(m.d, t, block);
        Stage<TG, kTokens>::prefetch(m.z, t, block);
        if constexpr (BETA) Stage<TG, kTokens>::prefetch(m.y, t, block);
    }

    static __device__ __forceinline__ float2 first_state(const Args &p, const Tokens &tok, int k, int c) {
        const int row = __shfl_sync(0xffffffffu, tok.row, k);
        return p.init ? load_state(p.init + (size_t)row * p.D, c, p.D) : splat(0.f);
    }
    static __device__ __forceinline__ float2 last_gradient(const GradArgs &q, const Tokens &tok, int k, int c) {
        const int row = __shfl_sync(0xffffffffu, tok.row, k);
        return q.dfin ? load_state(q.dfin + (size_t)row * q.f.D, c, q.f.D) : splat(0.f);
    }

    // What a warp keeps of its tokens' gates between the walks (the compiler drops what
    // the arm at hand does not have).
    struct Held {
        float2 a[kTokens], n[kTokens], i[kTokens], soft[kTokens];
    };

    // The gates of the warp's tokens and its maps, (R, H) and C.  PLAIN: all of them
    // inside one request, neither its first nor its last token among them, and their channels
    // whole words where they are stored as such.
    template <bool PLAIN>
    static __device__ __forceinline__ void first_walk(const GradArgs &q, const Input &in, const Tokens &tok, int c,
                                                      int lane, float2 bias, float2 scale, Held &held, float2 &R,
                                                      float2 &H, float2 &C) {
        const Args &p = q.f;
        float2 sum = splat(0.f);
        H = splat(0.f), C = splat(0.f);
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            float2 y = splat(0.f);
            if constexpr (BETA) y = in.y[0].at(k, lane);
            const Gates g = token_gates<RAW, BETA, MODE>(in.z.at(k, lane), y, bias, scale, p.sigmoid);
            held.a[k] = g.a, held.n[k] = g.n, held.i[k] = g.i, held.soft[k] = g.soft;
            float2 u = scaled<BETA, MODE>(in.x.at(k, lane), g.n, g.i), own_g = g.g;
            if (!PLAIN) {
                if (!(tok.own >> k & 1u)) held.a[k] = splat(1.f), own_g = u = splat(0.f);
                if (tok.first >> k & 1u) H = first_state(p, tok, k, c);
            }
            H = fma2(held.a[k], H, u);
            sum = sum + own_g;
        }
#pragma unroll
        for (int k = kTokens - 1; k >= 0; --k) {
            float2 d = in.d.at(k, lane);
            if (!PLAIN) {
                if (!(tok.own >> k & 1u)) d = splat(0.f);
                if (tok.last >> k & 1u) d = d + last_gradient(q, tok, k, c);
            }
            C = held.a[k] * (d + C);
            if (!PLAIN && (tok.first >> k & 1u)) C = splat(0.f);
        }
        R = !PLAIN && tok.first ? splat(kBegins) : root_of(sum);
    }

    // The gradients of the warp's tokens, from the state before and c behind them.
    template <bool PLAIN>
    static __device__ __forceinline__ void second_walk(const GradArgs &q, const GradMaps &m, Input &in,
                                                       const Tokens &tok, int t, int c, int lane, float2 scale,
                                                       const Held &held, float2 h, float2 dc, Sums &sums) {
        const Args &p = q.f;
        float2 prev[kTokens];
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            if (!PLAIN && (tok.first >> k & 1u)) h = first_state(p, tok, k, c);
            prev[k] = h;
            if (PLAIN || (tok.own >> k & 1u))
                h = fma2(held.a[k], h, scaled<BETA, MODE>(in.x.at(k, lane), held.n[k], held.i[k]));
        }
        const int first = c - 2 * lane, n_row = p.D - first;  // of the block's channels
#pragma unroll
        for (int k = kTokens - 1; k >= 0; --k) {
            if (!PLAIN && !(tok.own >> k & 1u)) continue;  // hands c on
            const float2 a = held.a[k], n = held.n[k], i = held.i[k];
            float2 dh = in.d.at(k, lane) + dc;
            if (!PLAIN && (tok.last >> k & 1u)) dh = dh + last_gradient(q, tok, k, c);
            const float2 x = in.x.at(k, lane);
            dc = a * dh;
            float2 d = dc * prev[k];
            if (MODE != kNone) {  // n'(g) i x dh
                float2 w = dh * x;
                if (BETA) w = w * i;
                if (MODE == kLerp) {
                    d = fma2(w, -a, d);
                } else {  // n' = -a^2 / n; where n is 0 (a >= 1) it is taken as 0
                    const float2 r = make_float2(n.x > 0.f ? reciprocal(n.x) : 0.f, n.y > 0.f ? reciprocal(n.y) : 0.f);
                    d = fma2(w, -(a * a * r), d);
                }
            }
            if (RAW) {  // sigmoid(z) = 1 - e^-softplus(z)
                sums.scale = fma2(d, held.soft[k], sums.scale);
                d = d * (-scale * exponential(-held.soft[k]).m);
                sums.bias = sums.bias + d;
            }
            const float2 w = MODE == kNone ? dh : n * dh, dx = BETA ? w * i : w;
            float2 dy = splat(0.f);
            if (BETA) {
                dy = w * x;
                if (p.sigmoid) dy = dy * fma2(i, -i, i);
            }
            if (PLAIN && WIDE) {
                in.x.v[k][lane] = pack<TA>(dx);
                in.z.v[k][lane] = pack<TG>(d);
                if constexpr (BETA) in.y[0].v[k][lane] = pack<TG>(dy);
            } else {
                store_row<TA>(static_cast<TA *>(q.dx) + (t + k) * q.dxs + first, dx, lane, n_row);
                store_row<TG>(static_cast<TG *>(q.dg) + (t + k) * q.dgs + first, d, lane, n_row);
                if constexpr (BETA) store_row<TG>(static_cast<TG *>(q.db) + (t + k) * q.dbs + first, dy, lane, n_row);
            }
            if (!PLAIN && (tok.first >> k & 1u)) {
                const int row = __shfl_sync(0xffffffffu, tok.row, k);
                if (q.dinit) store_state(q.dinit + (size_t)row * p.D, c, p.D, dc);
                dc = splat(0.f);
            }
        }
        if (PLAIN && WIDE) {
            ptx::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                ptx::tma_store_2d(&m.dx, c, t, in.x.v);
                ptx::tma_store_2d(&m.dz, c, t, in.z.v);
                if constexpr (BETA) ptx::tma_store_2d(&m.dy, c, t, in.y[0].v);
                ptx::bulk_commit();
            }
        }
    }

    static __device__ __forceinline__ void run(const GradArgs &q, const GradMaps &m, Shared &s) {
        const Args &p = q.f;
        Rest &r = s.r;
        const Place at = place_of(p);
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int block = (int)(blockIdx.x / at.size), c = block * 64 + 2 * lane;
        constexpr unsigned kAll = (1u << kTokens) - 1u;
        const int window = at.S * kTile, steps = windows(at, window);
        if (lane == 0) {
            ptx::mbar_init(&r.bar[warp][0], 1);
            ptx::mbar_init(&r.bar[warp][1], 1);
            ptx::fence_mbar_init();
        }
        __syncwarp();
        ptx::grid_wait();
        // the windows from the last to the first
        int t = at.base + (steps - 1) * window + at.rank * kTile + warp * kTokens;
        Seen seen;
        Tokens tok = {}, next = {};
        if (steps > 0) {
            tok = look_up(p, at.lo, at.hi, t, kTokens, lane, seen);
            fill(q, m, s.in[warp][0], &r.bar[warp][0], t, window, block, tok.own, lane);
        }
        float2 bias = splat(0.f), scale = bias;
        if (RAW) bias = load_state(p.bias, c, p.D), scale = load_state(p.scale, c, p.D);
        if (at.size > 1) exchange_init(r.x);
        gradient_duties(q, at.size * kWarps, at.me * kWarps + warp, lane, c, blockIdx.x < at.size);

        const bool whole = !WIDE || (whole_words<TA>(p.D, block) && whole_words<TG>(p.D, block));
        Sums sums = {};
        float carry = 0.f;  // c of this thread's channel (see Meet) behind the window
        for (int turn = 0; turn < steps; ++turn, t -= window) {
            const int stage = turn % kRing;
            Input &in = s.in[warp][stage];
            if (kRing == 2 && WIDE && turn + 1 < steps) {
                next = look_up(p, at.lo, at.hi, t - window, kTokens, lane, seen);
                if (lane == 0) ptx::bulk_wait_read();  // the other stage's gradients have left it
                __syncwarp();
                fill(q, m, s.in[warp][stage ^ 1], &r.bar[warp][stage ^ 1], t - window, window, block, next.own, lane);
            }
            if (kRing == 1 && turn + 1 < steps && WIDE && lane == 0) prefetch(m, t - window, block);
            // the state that the forward pass kept before the tile, early
            const int tile = t - warp * kTokens, ch = block * 64 + (threadIdx.x & 63);
            float kept = 0.f;
            if (tile < at.hi && ch < p.D)
                kept = p.chunk[(size_t)(tile / kChunk) * p.D + ch];
            if (WIDE) {
                if (!ptx::mbar_wait(&r.bar[warp][stage], turn / kRing & 1) && p.err) atomicOr(p.err, kErrTimeout);
            } else {
                __syncwarp();
            }
            const bool plain = tok.own == kAll && !(tok.first | tok.last) && whole;
            Held held;
            float2 R, H, C;
            if (plain) first_walk<true>(q, in, tok, c, lane, bias, scale, held, R, H, C);
            else first_walk<false>(q, in, tok, c, lane, bias, scale, held, R, H, C);
            *reinterpret_cast<float4 *>(&r.fwd[warp][2 * lane]) = make_float4(R.x, H.x, R.y, H.y);
            *reinterpret_cast<float4 *>(&r.rev.map[warp][2 * lane]) = make_float4(R.x, C.x, R.y, C.y);
            __syncthreads();
            Meet<true, kWarps> meet;
            const float2 whole = meet.send(r.rev, r.x, at, turn);
            {  // while the maps are on their way: the states before the warps' runs
                float h = kept;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    if (w / meet.kMine == meet.part) r.h[w][meet.c] = h;
                    h = apply(r.fwd[w][meet.c], h);
                }
            }
            meet.receive(r.rev, r.x, at, turn, whole, carry, p.err);
            __syncthreads();
            const float2 dc = *reinterpret_cast<const float2 *>(&r.rev.h[warp][2 * lane]);
            const float2 h = *reinterpret_cast<const float2 *>(&r.h[warp][2 * lane]);
            if (plain) second_walk<true>(q, m, in, tok, t, c, lane, scale, held, h, dc, sums);
            else second_walk<false>(q, m, in, tok, t, c, lane, scale, held, h, dc, sums);
            if ((kRing == 1 || !WIDE) && turn + 1 < steps) {
                next = look_up(p, at.lo, at.hi, t - window, kTokens, lane, seen);
                if (lane == 0) ptx::bulk_wait_read();
                __syncwarp();
                fill(q, m, s.in[warp][(turn + 1) % kRing], &r.bar[warp][0], t - window, window, block, next.own, lane);
            }
            tok = next;
        }
        if (lane == 0) ptx::bulk_wait();
        if (RAW) {  // sums over the block's warps, then over the cluster's blocks
            __syncthreads();
            *reinterpret_cast<float4 *>(&r.fwd[warp][2 * lane]) =
                make_float4(sums.bias.x, sums.scale.x, sums.bias.y, sums.scale.y);
            __syncthreads();
            if (at.size > 1) {  // no group uses its buffers any more
                cluster_arrive();
                cluster_wait();
            }
            if (threadIdx.x < 64) {
                const int k = threadIdx.x, ch = block * 64 + k;
                float2 v = r.fwd[0][k];
                for (int w = 1; w < kWarps; ++w) v = v + r.fwd[w][k];
                if (at.size > 1) {
                    if (at.me == 0 && k == 0) exchange_expect(r.x, 2, at.size);
                    exchange_send(r.x, 0, 2, at.me, 0, k, v);
                    if (at.me == 0) {
                        if (!ptx::mbar_wait(&r.x.bar[2], 0, 1u << 20) && p.err) atomicOr(p.err, kErrTimeout);
                        v = r.x.map[0][0][k];
                        for (int i = 1; i < at.size; ++i) v = v + r.x.map[0][i][k];
                    }
                }
                if (at.me == 0 && ch < p.D) {
                    if (q.dbias) q.dbias[ch] = v.x;
                    if (q.dscale) q.dscale[ch] = v.y;
                }
            }
        }
        if (at.size > 1) {  // no block leaves while another may still send to it
            cluster_arrive();
            cluster_wait();
        }
    }
};

template <bool WIDE, typename TA, typename TG, bool RAW, bool BETA, int MODE>
__global__ void __launch_bounds__(kWarps * 32, 2) scan_grad_kernel(const __grid_constant__ GradArgs q,
                                                                  const __grid_constant__ GradMaps m) {
    using G = Backward<WIDE, TA, TG, RAW, BETA, MODE>;
    extern __shared__ __align__(128) unsigned char smem[];
    G::run(q, m, *reinterpret_cast<typename G::Shared *>(smem));
}

template <bool WIDE, typename TA, typename TG, bool RAW, bool BETA, int MODE>
cudaError_t launch_grad_one(const GradArgs &args, cudaStream_t stream) {
    using G = Backward<WIDE, TA, TG, RAW, BETA, MODE>;
    auto kernel = scan_grad_kernel<WIDE, TA, TG, RAW, BETA, MODE>;
    GradArgs q = args;
    const Args &p = q.f;
    const int cb = (p.D + 63) / 64;
    int S = 1;
    const cudaError_t e =
        cluster_blocks((const void *)kernel, kWarps, sizeof(typename G::Shared), cb, (p.T + G::kTile - 1) / G::kTile, &S);
    if (e != cudaSuccess) return e;
    share_out(q.f, S, G::kTile);
    GradMaps m = {};
    constexpr int ta = type_of<TA>(), tg = type_of<TG>(), n = G::kTokens;
    if (WIDE && !(make_token_map(&m.x, p.x, ta, p.xs, p.D, p.T, n) &&
                    make_token_map(&m.d, q.d_o, ta, q.dos, p.D, p.T, n) &&
                    make_token_map(&m.z, p.decay, tg, p.gs, p.D, p.T, n) &&
                    make_token_map(&m.dx, q.dx, ta, q.dxs, p.D, p.T, n) &&
                    make_token_map(&m.dz, q.dg, tg, q.dgs, p.D, p.T, n) &&
                    (!BETA || (make_token_map(&m.y, p.beta, tg, p.bs, p.D, p.T, n) &&
                               make_token_map(&m.dy, q.db, tg, q.dbs, p.D, p.T, n)))))
        return cudaErrorInvalidValue;
    return launch_clusters(cb, S, kWarps, sizeof(typename G::Shared), true, stream, kernel, q, m);
}

template <bool WIDE, typename TA, typename TG, bool RAW, bool BETA>
cudaError_t launch_grad_mode(const GradArgs &q, cudaStream_t stream) {
    if (q.f.mode == kNone) return launch_grad_one<WIDE, TA, TG, RAW, BETA, kNone>(q, stream);
    if (q.f.mode == kLerp) return launch_grad_one<WIDE, TA, TG, RAW, BETA, kLerp>(q, stream);
    return launch_grad_one<WIDE, TA, TG, RAW, BETA, kUnit>(q, stream);
}

template <bool WIDE, typename TA, typename TG>
cudaError_t launch_grad_types(const GradArgs &q, cudaStream_t stream) {
    if (q.f.bias)
        return q.f.beta ? launch_grad_mode<WIDE, TA, TG, true, true>(q, stream)
                        : launch_grad_mode<WIDE, TA, TG, true, false>(q, stream);
    return q.f.beta ? launch_grad_mode<WIDE, TA, TG, false, true>(q, stream)
                    : launch_grad_mode<WIDE, TA, TG, false, false>(q, stream);
}

}  // namespace scan
}  // namespace gdn
