// scan_cluster.cuh -- what gdn_scan and its gradient share: clusters of blocks
// along time, maps of runs of tokens, the launch.
#pragma once

#include <cuda.h>  // CUtensorMap

#include <stddef.h>

#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "scan_launch.h"

namespace gdn {
namespace scan {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// All blocks of the cluster have come here.  Orders no memory accesses.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
constexpr int kMaxCluster = 16;
constexpr int kMaxWindow = kMaxCluster * 128;  // tokens that a cluster takes at a time, at most

// (R, H) of a run of one channel: it takes h to R^2 h + H, R^2 being the product of its a.
// That product itself may leave fp32's range both ways (128 tokens of |g| = 0.7), and a state
// that it multiplies come back into range: gates above 0 grow states that are zero or
// small, and what they have grown is forgotten again.  Its root, multiplied by twice, is in
// range wherever the result is; where it would not be it stops at 2^127, so that a state of
// zero stays one.  (With the product a window of 16-bit gates of 1 turned zeros to NaN.  The
// root costs 16384 x 4096 ragged fp16 163 us for 158, a training pass of 4 x 8192 x 2048
// bf16 466 for 461, and halves the error of long memories.)
// A run in which a request begins has R = -0 and takes nothing of what is before it, not
// even a NaN or an infinity (every other R is +0 at least).
constexpr float kBegins = -0.f, kLargest = 0x1p127f;
__device__ __forceinline__ bool begins(float R) { return __float_as_uint(R) == 0x80000000u; }
// What the run makes of the state h, if no request begins in it, and if one may.
__device__ __forceinline__ float pass(float2 r, float h) { return fmaf(h * r.x, r.x, r.y); }
__device__ __forceinline__ float apply(float2 r, float h) { return begins(r.x) ? r.y : pass(r, h); }
// The run k followed by r, the same two ways.
__device__ __forceinline__ float2 follow(float2 k, float2 r) {
    return make_float2(fminf(k.x * r.x, kLargest), pass(r, k.y));
}
__device__ __forceinline__ float2 fold(float2 k, float2 r) {
    return make_float2(begins(k.x) || begins(r.x) ? kBegins : fminf(k.x * r.x, kLargest), apply(r, k.y));
}
// R of a run whose g add up to sum: without a bias near 1, where runs are many.
__device__ __forceinline__ float2 root_of(float2 sum) {
    constexpr float kLog = 88.02969f;  // log of kLargest
    return exponential(make_float2(fminf(0.5f * sum.x, kLog), fminf(0.5f * sum.y, kLog))).a;
}

// ---------------------------------------------------------------- staging
// A warp's tokens of one tensor wait in shared memory of its own: TOKENS rows of 64
// channels.  Rows that begin on 16-byte addresses are one box of a tensor map, which
// completes on the warp's mbarrier (by cp.async, 16 bytes a lane, a warp was held up
// 160 cycles a copy).  Others are read by 4-byte words, which are shifted together
// where a 16-bit row begins between two words, after a prefetch to L2 a window
// earlier; tiles whose words would reach past the tensor's ends, channel by channel.
// (Bulk copies of the words of 16 bytes that such rows touch, shifted when they are
// read, were slower: 250 us for 16384 x 2046 bf16.)
template <typename T, int TOKENS>
struct alignas(128) Stage {
    static constexpr int kRow = 64 * (int)sizeof(T);
    static constexpr uint32_t kBytes = TOKENS * kRow;
    pair_t<T> v[TOKENS][32];

    __device__ __forceinline__ void fill(const CUtensorMap &map, int t, int block, uint64_t *bar) {
        ptx::tma_load_2d(v, &map, block * 64, t, bar);
    }
    static __device__ __forceinline__ void prefetch(const CUtensorMap &map, int t, int block) {
        ptx::tma_prefetch_2d(&map, block * 64, t);
    }
    // Token t + lane's row on its way to L2.
    static __device__ __forceinline__ void prefetch_row(const void *base, int64_t stride, int t, int end, int block,
                                                        int D, int lane) {
        const char *row = static_cast<const char *>(base) + ((int64_t)(t + lane) * stride + block * 64) * (int)sizeof(T);
        const int left = (D - block * 64) * (int)sizeof(T);
        if (lane >= TOKENS || t + lane >= end || left <= 0) return;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
        if (left > 128 && kRow > 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + 128));
    }
    __device__ __forceinline__ void fill_words(const void *base, int64_t stride, int t, int block, unsigned own, int D,
                                               int lane) {
        const T *row = static_cast<const T *>(base) + (int64_t)t * stride + block * 64;
        const int n = D - block * 64 < 64 ? D - block * 64 : 64;
        pair_t<T> r[TOKENS];  // all on their way before the first is stored
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int k = 0; k < TOKENS; ++k) {
                const bool on = own >> k & 1u;
                r[k].x = on && 2 * lane < n ? row[k * stride + 2 * lane] : 0.f;
                r[k].y = on && 2 * lane + 1 < n ? row[k * stride + 2 * lane + 1] : 0.f;
            }
        } else {
            const uintptr_t first = reinterpret_cast<uintptr_t>(row);
            const bool odd = stride & 1;
            if (!odd && !(first & 2u)) {  // no row begins between words
#pragma unroll
                for (int k = 0; k < TOKENS; ++k) {
                    const bool on = own >> k & 1u && 2 * lane < n;
                    r[k] = on ? reinterpret_cast<const uint32_t *>(row + k * stride)[lane] : 0u;
                }
            } else {
                // of two rows in turn both or one; the word behind lane 31's comes with a
                // load of its own
                uint32_t last[TOKENS];
#pragma unroll
                for (int k = 0; k < TOKENS; ++k) {
                    const bool split = ((first >> 1) + (odd ? k : 0)) & 1u, on = own >> k & 1u;
                    const uint32_t *w = reinterpret_cast<const uint32_t *>(row + k * stride - (split ? 1 : 0)) + lane;
                    r[k] = on && 2 * lane < n + (split ? 1 : 0) ? *w : 0u;
                    last[k] = on && split && lane == 31 && n == 64 ? w[1] : 0u;
                }
#pragma unroll
                for (int k = 0; k < TOKENS; ++k) {
                    const bool split = ((first >> 1) + (odd ? k : 0)) & 1u;
                    const uint32_t next = __shfl_down_sync(0xffffffffu, r[k], 1);
                    if (split) r[k] = __funnelshift_r(r[k], lane == 31 ? last[k] : next, 16);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < TOKENS; ++k) v[k][lane] = r[k];
    }
    __device__ __forceinline__ void fill_each(const void *base, int64_t stride, int t, int block, unsigned own, int D,
                                              int lane) {
        const int c = block * 64 + 2 * lane;
        const T *p = static_cast<const T *>(base) + (int64_t)t * stride + c;
        if (c >= D) own = 0u;
        pair_t<T> r[TOKENS];
#pragma unroll
        for (int k = 0; k < TOKENS; ++k)
            r[k] = (own >> k & 1u) ? load_pair<T>(p + k * stride, c + 1 < D) : zero_pair<T>();
#pragma unroll
        for (int k = 0; k < TOKENS; ++k) v[k][lane] = r[k];
    }
    __device__ __forceinline__ float2 at(int k, int lane) const { return unpack<T>(v[k][lane]); }
};
// Whether the words that a tile's rows touch lie inside the tensor.
__device__ __forceinline__ bool inside(const Args &p, int t, int tokens, int block) {
    return !(t == 0 && block == 0) && !(t + tokens >= p.T && (block + 1) * 64 >= p.D);
}

// Whether the block's channels end on a 16-byte boundary: a bulk store of a box that ends
// inside one writes the rest of it too, over what lies behind the row's channels there.
template <typename T>
__device__ __forceinline__ bool whole_words(int D, int block) {
    return (block + 1) * 64 <= D || D * (int)sizeof(T) % 16 == 0;
}

// [rows, channels] of elements of type T, boxes of 64 channels x `tokens` rows.
bool make_token_map(CUtensorMap *m, const void *base, int type, int64_t stride, int channels, int rows, int tokens);

// The exchange of the blocks' maps, one a window: a block sends its own to every
// block of its group by asynchronous stores that count on the receiver's
// mbarrier.  Nothing is fenced: a release at cluster scope would wait for the
// outputs that the block has just stored to HBM.  Two buffers in turn suffice: a
// block sends for window i + 2 once it has every block's map of window i + 1, which
// a block sends after it has read those of window i.
struct alignas(16) Exchange {
    float2 map[2][kMaxCluster][64];
    uint64_t bar[3];  // of the two buffers; of what the gradient sends at its end
};
__device__ __forceinline__ void exchange_init(Exchange &x) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) ptx::mbar_init(&x.bar[i], 1);
        ptx::fence_mbar_init();
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// One thread, once a window, before it waits for `n` blocks.
__device__ __forceinline__ void exchange_expect(Exchange &x, int bar, int n) {
    ptx::mbar_arrive_expect_tx(&x.bar[bar], (uint32_t)n * 64u * sizeof(float2));
}
// Sends channel c's v to block `to` of the cluster, in place `from` of buffer `par`.
__device__ __forceinline__ void exchange_send(Exchange &x, int par, int bar, int from, int to, int c, float2 v) {
    uint32_t base;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(base) : "r"(ptx::smem_u32(&x)), "r"(to));
    const uint32_t at = base + (uint32_t)offsetof(Exchange, map) + ((par * kMaxCluster + from) * 64 + c) * 8u;
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at),
                 "f"(v.x), "f"(v.y), "r"(base + (uint32_t)offsetof(Exchange, bar) + bar * 8u)
                 : "memory");
}
// Waits for the maps of the window that uses this buffer for the n-th time (from 0).
// The wait is bounded; a block that gave up goes on (with wrong results, reported),
// so that the others' stores still find its memory.
__device__ __forceinline__ void exchange_wait(Exchange &x, int par, int n, int32_t *err) {
    if (!ptx::mbar_wait(&x.bar[par], n & 1, 1u << 20) && err) atomicOr(err, kErrTimeout);
}

// A block's place in its cluster: group `group` of requests, whose tokens are
// [lo, hi), is walked by S blocks, of which this is number `rank` and the first is
// block `lead` of the cluster.  Windows begin at `base`, where the forward pass keeps
// a state.
struct Place {
    int size, me, S, rank, lead, lo, hi, base;
};
__device__ __forceinline__ Place place_of(const Args &p) {
    Place a;
    a.size = cluster_size(), a.me = cluster_rank();
    a.S = a.size / p.groups;
    const int group = a.me / a.S;
    a.rank = a.me - group * a.S, a.lead = group * a.S;
    a.lo = 0, a.hi = p.T;
    if (p.groups > 1) {
        const int first = group * p.per, end = first + p.per;
        a.lo = (first < p.B ? first : p.B) * p.L;
        a.hi = (end < p.B ? end : p.B) * p.L;
    }
    a.base = a.lo / kChunk * kChunk;
    return a;
}
__device__ __forceinline__ int windows(const Place &a, int window) {
    return a.hi > a.lo ? (a.hi - a.base + window - 1) / window : 0;
}

// The maps of a block's warps, of 64 channels each, and the states before their runs.
template <int WARPS>
struct alignas(16) Meeting {  // a warp writes its maps 16 bytes a lane
    float2 map[WARPS][64];
    float h[WARPS][64];
};
// Between two barriers of the block its threads turn the warps' maps into the
// states before the warps' runs: a thread takes one channel, for two of the warps.
// Every thread folds all maps of its channel itself: with 64 threads doing it for the
// block, the others waited 3,100 cycles a window of 8 blocks for 300 dependent
// instructions.  Warps and blocks follow one another upwards, or (REVERSE) downwards.
template <bool REVERSE, int WARPS>
struct Meet {
    static constexpr int kParts = WARPS * 32 / 64, kMine = WARPS / kParts;
    int c, part;
    float2 before[kMine];  // the run before each of this thread's warps

    // First: the block's map, to every block of its group.
    __device__ __forceinline__ float2 send(const Meeting<WARPS> &m, Exchange &x, const Place &at, int turn) {
        c = threadIdx.x & 63, part = threadIdx.x >> 6;
        float2 run = make_float2(1.f, 0.f);
        uint32_t any = 0u;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            const float2 k = m.map[REVERSE ? WARPS - 1 - i : i][c];
            if (i / kMine == part) before[i % kMine] = run;
            any |= __float_as_uint(k.x);
            run = follow(run, k);
        }
        if (any >> 31) {  // a request begins in one of them
            run = make_float2(1.f, 0.f);
            for (int i = 0; i < WARPS; ++i) {
                const float2 k = m.map[REVERSE ? WARPS - 1 - i : i][c];
#pragma unroll
                for (int j = 0; j < kMine; ++j)
                    if (i == part * kMine + j) before[j] = run;
                run = fold(run, k);
            }
        }
        if (at.S > 1) {
            const int par = turn & 1;
            if (threadIdx.x == 0) exchange_expect(x, par, at.S);
            for (int r = part; r < at.S; r += kParts) exchange_send(x, par, par, at.rank, at.lead + r, c, run);
        }
        return run;
    }
    // Then: the states before the runs, from `carry`, the one before the window,
    // which moves on by a window.
    __device__ __forceinline__ void receive(Meeting<WARPS> &m, Exchange &x, const Place &at, int turn, float2 run,
                                            float &carry, int32_t *err) {
        float h = carry;
        const int S = at.S, rank = at.rank;
        if (S > 1) {
            const int par = turn & 1;
            exchange_wait(x, par, turn >> 1, err);
            const float2 *map = &x.map[par][REVERSE ? S - 1 : 0][c];
            constexpr int kNext = REVERSE ? -64 : 64;
            const int me = REVERSE ? S - 1 - rank : rank;
            const float c0 = carry;
            uint32_t any = 0u;
#pragma unroll 4
            for (int i = 0; i < S; ++i) {
                const float2 k = map[i * kNext];
                if (i == me) h = carry;
                any |= __float_as_uint(k.x);
                carry = pass(k, carry);
            }
            if (any >> 31) {
                carry = c0;
                for (int i = 0; i < S; ++i) {
                    if (i == me) h = carry;
                    carry = apply(map[i * kNext], carry);
                }
            }
        } else {
            carry = apply(run, carry);
        }
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int w = part * kMine + j;
            m.h[REVERSE ? WARPS - 1 - w : w][c] = apply(before[j], h);
        }
    }
};

// The blocks along time of one channel block: the most, up to a cluster's limit,
// with which all clusters are resident at once, and no more than there are tiles.
inline cudaError_t cluster_blocks(const void *kernel, int warps, size_t smem, int channel_blocks, int tiles, int *S) {
    cudaError_t e = smem_attr(kernel, (int)smem);
    if (e == cudaSuccess) e = large_clusters(kernel);
    int s = tiles < kMaxCluster ? tiles : kMaxCluster, n = 0;
    if (e == cudaSuccess && s > 1) {
        e = resident_clusters(kernel, warps * 32, smem, 1, &n);
        if (s > n / channel_blocks) s = n / channel_blocks;
    }
    for (; e == cudaSuccess && s > 1; --s) {
        e = resident_clusters(kernel, warps * 32, smem, s, &n);
        if (n >= channel_blocks) break;
    }
    *S = s < 1 ? 1 : s;
    return e;
}

// Requests of equal rows are independent chains, so a cluster of `size` blocks may
// take groups of them side by side, each with fewer blocks: the exchange then joins
// fewer of them.  As many groups as keep the number of windows within an eighth (rows
// that do not share out evenly, tiles that two groups cut).  4 x 8192 x 2048 bf16 in
// clusters of 8: in four groups 142 us, in one 162 us; its training pass 466 and 539.
inline void share_out(Args &p, int size, int tile) {
    p.groups = 1, p.per = p.B;
    if (p.cu || p.B < 2) return;
    auto steps = [&](int64_t tokens, int blocks) { return (tokens + (int64_t)blocks * tile - 1) / (blocks * tile); };
    const int64_t one = steps(p.T, size);
    for (int g = p.B < size ? p.B : size; g > 1; --g) {
        if (size % g) continue;
        const int per = (p.B + g - 1) / g;
        const int64_t tokens = (int64_t)per * p.L, cut = tokens % kChunk ? kChunk : 0;
        if (steps(tokens + cut, size / g) * 8 <= one * 9) {
            p.groups = g, p.per = per;
            return;
        }
    }
}

// Launches a kernel in clusters of S blocks; `early`: as launch_early().
template <typename... P, typename... A>
cudaError_t launch_clusters(int channel_blocks, int S, int warps, size_t smem, bool early, cudaStream_t stream,
                            void (*kernel)(P...), const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)channel_blocks * (unsigned)S);
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = early ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
constexpr int type_of() {
    return std::is_same<T, float>::value ? 0 : (std::is_same<T, __half>::value ? 1 : 2);
}

}  // namespace scan
}  // namespace gdn
