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

// (A, H) of a run of two channels: x, y the A of both, z, w the H.  A run in which
// a request begins has A = -0 and takes nothing of what is before it, not even a
// NaN or an infinity (every other A is a product of exponentials, +0 at least).
constexpr float kBegins = -0.f;
__device__ __forceinline__ float4 map_of(float2 A, float2 H) { return make_float4(A.x, A.y, H.x, H.y); }
__device__ __forceinline__ float2 map_a(const float4 r) { return make_float2(r.x, r.y); }
__device__ __forceinline__ float2 map_h(const float4 r) { return make_float2(r.z, r.w); }
__device__ __forceinline__ bool begins(const float4 r) { return __float_as_uint(r.x) == 0x80000000u; }
// The run (A, H) followed by r.  RESETS: a request may begin in r.
template <bool RESETS>
__device__ __forceinline__ void fold(float2 &A, float2 &H, const float4 r) {
    const float2 h = fma2(map_a(r), H, map_h(r)), a = A * map_a(r);
    if (RESETS && begins(r)) {
        A = map_a(r);
        H = map_h(r);
    } else {
        const bool b = RESETS && __float_as_uint(A.x) == 0x80000000u;
        A = b ? A : a;
        H = h;
    }
}
__device__ __forceinline__ float2 apply(const float4 r, float2 h) {
    const float2 v = fma2(map_a(r), h, map_h(r));
    return begins(r) ? map_h(r) : v;
}

// The state after the runs r[0], r[32], ... r[32 (n - 1)] of a lane, and in `at` the
// one before run `me`.  Four maps are on their way at a time.
__device__ __forceinline__ float2 apply_all(const float4 *r, int n, int me, float2 h, float2 &at) {
    const float2 h0 = h;
    uint32_t any = 0u;
    for (int i = 0; i < n; i += 4) {
        float4 k[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = r[32 * (i + j < n ? i + j : n - 1)];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (i + j >= n) break;
            if (i + j == me) at = h;
            any |= __float_as_uint(k[j].x);
            h = fma2(map_a(k[j]), h, map_h(k[j]));
        }
    }
    if (any >> 31) {  // a request begins in one of them
        h = h0;
        for (int i = 0; i < n; ++i) {
            const float4 k = r[32 * i];
            if (i == me) at = h;
            h = __float_as_uint(k.x) >> 31 ? map_h(k) : fma2(map_a(k), h, map_h(k));
        }
    }
    return h;
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
// outputs that the block has just stored to HBM (measured: 3.9 us a window with a
// cluster barrier in place of this, 16 warps an SM).  Two buffers in turn suffice:
// a block sends for window i + 2 once it has every block's map of window i + 1,
// which a block sends after all its warps have read those of window i.
struct Exchange {
    float4 map[2][kMaxCluster][32];
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
    ptx::mbar_arrive_expect_tx(&x.bar[par], (uint32_t)S * 32u * sizeof(float4));
}
// A warp sends v (a lane's two channels) to block `to`, in this block's place.
__device__ __forceinline__ void exchange_send(Exchange &x, int par, int from, int to, int lane, float4 v) {
    uint32_t at, bar;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(&x.map[par][from][lane])), "r"(to));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(ptx::smem_u32(&x.bar[par])), "r"(to));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
                 : "memory");
}
// Waits for the maps of the window that uses this buffer for the n-th time (from 0).
// The wait is bounded; a block that gave up goes on (with wrong results, reported),
// so that the others' stores still find its memory.
__device__ __forceinline__ void exchange_wait(Exchange &x, int par, int n, int32_t *err) {
    if (!ptx::mbar_wait(&x.bar[par], n & 1, 1u << 20) && err) atomicOr(err, kErrTimeout);
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
