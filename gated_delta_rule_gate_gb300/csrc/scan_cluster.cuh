// scan_cluster.cuh -- what gdn_scan and its gradient share: clusters of blocks
// along time, maps of runs of tokens, the launch.
#pragma once

#include <cuda.h>  // CUtensorMap

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
constexpr int kWarps = 8;
constexpr int kMaxCluster = 16;

// (A, H) of a run of one channel.  A run in which a request begins has A = -0 and
// takes nothing of what is before it, not even a NaN or an infinity (every other A
// is a product of exponentials, +0 at least).
constexpr float kBegins = -0.f;
__device__ __forceinline__ bool begins(float A) { return __float_as_uint(A) == 0x80000000u; }
// What the run makes of the state h.
__device__ __forceinline__ float apply(float2 r, float h) { return begins(r.x) ? r.y : fmaf(r.x, h, r.y); }
// The run k followed by r.
__device__ __forceinline__ float2 fold(float2 k, float2 r) {
    const float A = begins(k.x) ? kBegins : k.x * r.x;
    return make_float2(begins(r.x) ? kBegins : A, apply(r, k.y));
}

// ---------------------------------------------------------------- staging
// A warp's tokens of one tensor wait in shared memory of its own: TOKENS rows of 64
// channels, one box of a tensor map, which completes on the warp's mbarrier.  (By
// cp.async, 16 bytes a lane, a warp was held up 160 cycles a copy on the way.)
// Without a tensor map -- rows that do not begin on 16-byte addresses -- the lanes
// load their channels and store them here.
template <typename T, int TOKENS>
struct alignas(128) Stage {
    pair_t<T> v[TOKENS][32];
    static constexpr uint32_t kBytes = TOKENS * 64 * sizeof(T);

    __device__ __forceinline__ void fill(const CUtensorMap &map, int t, int block, uint64_t *bar) {
        ptx::tma_load_2d(&v[0][0], &map, block * 64, t, bar);
    }
    __device__ __forceinline__ void fill_plain(const void *base, int64_t stride, int t, int block, unsigned own, int D,
                                               bool vec, int lane) {
        const int c = block * 64 + 2 * lane;
        const T *p = static_cast<const T *>(base) + (int64_t)t * stride + c;
        if (c >= D) own = 0u;
#pragma unroll
        for (int k = 0; k < TOKENS; ++k)
            v[k][lane] = (own >> k & 1u) ? load_pair<T>(p + k * stride, vec, c + 1 < D) : zero_pair<T>();
    }
    __device__ __forceinline__ float2 at(int k, int lane) const { return unpack<T>(v[k][lane]); }
};

// [rows, channels] of elements of type T, boxes of 64 channels x `tokens` rows.
bool make_token_map(CUtensorMap *m, const void *base, int type, int64_t stride, int channels, int rows, int tokens);

// The exchange of the blocks' maps, one a window: a block sends its own to every
// block of the cluster by asynchronous stores that count on the receiver's
// mbarrier.  Nothing is fenced: a release at cluster scope would wait for the
// outputs that the block has just stored to HBM.  Two buffers in turn suffice: a
// block sends for window i + 2 once it has every block's map of window i + 1, which
// a block sends after it has read those of window i.
struct Exchange {
    float2 map[2][kMaxCluster][64];
    uint64_t bar[2];
};
__device__ __forceinline__ void exchange_init(Exchange &x) {
    if (threadIdx.x == 0) {
        ptx::mbar_init(&x.bar[0], 1);
        ptx::mbar_init(&x.bar[1], 1);
        ptx::fence_mbar_init();
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// One thread, once a window, before it waits.
__device__ __forceinline__ void exchange_expect(Exchange &x, int par, int S) {
    ptx::mbar_arrive_expect_tx(&x.bar[par], (uint32_t)S * 64u * sizeof(float2));
}
// Sends channel c's v to block `to`, in block `from`'s place.
__device__ __forceinline__ void exchange_send(Exchange &x, int par, int from, int to, int c, float2 v) {
    uint32_t at, bar;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(&x.map[par][from][c])), "r"(to));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(ptx::smem_u32(&x.bar[par])), "r"(to));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at),
                 "f"(v.x), "f"(v.y), "r"(bar)
                 : "memory");
}
// Waits for the maps of the window that uses this buffer for the n-th time (from 0).
// The wait is bounded; a block that gave up goes on (with wrong results, reported),
// so that the others' stores still find its memory.
__device__ __forceinline__ void exchange_wait(Exchange &x, int par, int n, int32_t *err) {
    if (!ptx::mbar_wait(&x.bar[par], n & 1, 1u << 20) && err) atomicOr(err, kErrTimeout);
}

// The maps of a block's warps, of 64 channels each, and the states before them.
struct Meeting {
    float2 map[kWarps][64];
    float h[kWarps][64];
};
// One of 64 threads, for channel c, between two barriers of the block: the states
// before the warps' runs, from `carry`, the state before the window, which moves on
// by a window.  Warps and blocks follow one another upwards, or (REVERSE) downwards.
// One thread a channel instead of every warp for itself: the maps are read once (the
// warps' own folding took 1,700 cycles a window of 8 blocks, of 6,800).
template <bool REVERSE>
__device__ __forceinline__ void meet(Meeting &m, Exchange &x, int S, int rank, int turn, int c, float &carry,
                                     int32_t *err) {
    const int par = turn & 1;
    float2 run = make_float2(1.f, 0.f);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        float2 *at = &m.map[REVERSE ? kWarps - 1 - i : i][c];
        const float2 k = *at;
        *at = run;
        run = fold(run, k);
    }
    float h = carry;
    if (S > 1) {
        if (c == 0) exchange_expect(x, par, S);
        for (int r = 0; r < S; ++r) exchange_send(x, par, rank, r, c, run);
        exchange_wait(x, par, turn >> 1, err);
        for (int i = 0; i < S; i += 4) {  // four maps on their way at a time
            float2 k[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = i + j < S ? i + j : S - 1;
                k[j] = x.map[par][REVERSE ? S - 1 - r : r][c];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (i + j >= S) break;
                if ((REVERSE ? S - 1 - (i + j) : i + j) == rank) h = carry;
                carry = apply(k[j], carry);
            }
        }
    } else {
        carry = apply(run, carry);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m.h[w][c] = apply(m.map[w][c], h);
}

// The blocks along time of one channel block: the most, up to a cluster's limit,
// with which all clusters are resident at once, and no more than there are tiles.
inline cudaError_t cluster_blocks(const void *kernel, size_t smem, int channel_blocks, int tiles, int *S) {
    cudaError_t e = smem_attr(kernel, (int)smem);
    if (e == cudaSuccess) e = large_clusters(kernel);
    int s = tiles < kMaxCluster ? tiles : kMaxCluster;
    for (; e == cudaSuccess && s > 1; --s) {
        int n = 0;
        e = resident_clusters(kernel, kWarps * 32, smem, s, &n);
        if (n >= channel_blocks) break;
    }
    *S = s < 1 ? 1 : s;
    return e;
}

// Launches a kernel in clusters of S blocks.
template <typename... P, typename... A>
cudaError_t launch_clusters(int channel_blocks, int S, size_t smem, cudaStream_t stream, void (*kernel)(P...),
                            const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)channel_blocks * (unsigned)S);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
constexpr int type_of() {
    return std::is_same<T, float>::value ? 0 : (std::is_same<T, __half>::value ? 1 : 2);
}

}  // namespace scan
}  // namespace gdn
