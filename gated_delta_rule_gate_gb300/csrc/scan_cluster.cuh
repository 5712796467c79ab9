// scan_cluster.cuh -- what gdn_scan and its gradient share: clusters of blocks
// along time, maps of runs of tokens, the launch.
#pragma once

#include "launch.h"
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
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Writes v to the same place of block `rank`'s shared memory.
__device__ __forceinline__ void store_remote(float4 *p, uint32_t rank, float4 v) {
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p)), to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

constexpr int kWarps = 8;
constexpr int kMaxCluster = 16;

// (A, H) of a run of two channels: x, y the first's, z, w the second's.  A run
// in which a request begins has A = -0 and takes nothing of what is before it,
// not even a NaN or an infinity (every other A is a product of exponentials, +0
// at least).  Both channels of a run agree on it.
constexpr float kBegins = -0.f;
__device__ __forceinline__ bool begins(const float4 r) { return __float_as_uint(r.x) == 0x80000000u; }
// k followed by r.
__device__ __forceinline__ void fold(float4 &k, const float4 r) {
    if (begins(r)) {
        k = r;
    } else {
        const bool b = begins(k);
        k.y = fmaf(r.x, k.y, r.y);
        k.x = b ? kBegins : k.x * r.x;
        k.w = fmaf(r.z, k.w, r.w);
        k.z *= r.z;
    }
}
__device__ __forceinline__ float2 apply(const float4 r, float2 h) {
    return begins(r) ? make_float2(r.y, r.w) : make_float2(fmaf(r.x, h.x, r.y), fmaf(r.z, h.y, r.w));
}

// The blocks along time of one channel block: the most, up to a cluster's limit,
// with which all clusters are resident at once, and no more than there are tiles.
inline int cluster_blocks(int channel_blocks, int tiles, int resident) {
    int S = 1;
    while (S < kMaxCluster && S < tiles && 2 * S * channel_blocks <= resident) S *= 2;
    return S;
}

// Launches a kernel in clusters of S blocks.
template <typename P>
cudaError_t launch_clusters(void (*kernel)(P), const P &p, int channel_blocks, int S, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)channel_blocks * (unsigned)S);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace scan
}  // namespace gdn
