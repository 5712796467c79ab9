// grad_clip.cu -- gdn_grad_clip: the norm over many tensors, and their scaling.
//
// Two kernels a group of tensors (up to kMany, whose table travels as a kernel
// argument, so nothing is copied to the device first): every block sums the
// squares of its chunks into one partial, and then every block adds up all
// partials in one order and scales its chunks.  Bound by HBM: the gradients are
// read for the norm and, since it has to be known first, once more to be scaled;
// the second kernel takes the chunks from the end, where the L2 still holds what
// the first one read last.  2^28 fp32 elements, out of place: 486 us, 6.6 TB/s.
// (One launch of a cluster of 16 blocks, for few and small tensors, took 14 to 25 us
// where the two kernels take 6 to 10.)
#include <math.h>

#include "launch.h"
#include "ptx.cuh"
#include "status.h"
#include "twofloat.cuh"
#include "values.cuh"

namespace gdn {
namespace clip {

constexpr int kThreads = 256;
constexpr int kBlocks = 152 * 8;
constexpr int kMany = 512;
// Elements that a block takes at a time: fewer of up to 2 M elements, so that they
// reach all SMs (us a call, out of place, chunks of 8192 / 2048: 0.26 M fp32 elements
// 6.9 / 5.9, 1.0 M 7.7 / 7.1, 2.1 M 11.6 / 8.1).
constexpr int kChunk = 8192, kSmallChunk = 2048;
constexpr int64_t kSmall = 1 << 21;

struct Tensor {
    const void *in;
    void *out;
    int64_t n;
    int32_t first;  // its first chunk, counted over the table
    int32_t type;   // gdn_dtype
};
template <int MAX>
struct Table {
    Tensor t[MAX];
    int count, chunks, chunk;  // tensors, chunks, elements of a chunk
};

template <int MAX>
__device__ __forceinline__ int find_tensor(const Table<MAX> &tab, int chunk) {
    int lo = 0, hi = tab.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.t[mid].first <= chunk) lo = mid; else hi = mid;
    }
    return lo;
}

// Elements before the first 16-byte address of p, of n.
template <typename T>
__device__ __forceinline__ int head_of(const T *p, int n) {
    const int head = (int)((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / sizeof(T));
    return head < n ? head : n;
}

// In words of 16 bytes, and one by one before and after them (2^28 bf16 elements from
// an odd address: 293 us with the result as far from one, 581 one by one; 252 from a
// 16-byte address).
template <int THREADS, typename T>
__device__ __forceinline__ float chunk_squares(const T *p, int n) {
    constexpr int V = sizeof(T) == 4 ? 4 : 8;
    const int head = head_of(p, n), end = head + (n - head) / V * V;
    float part[V] = {};
#pragma unroll 4
    for (int i = head + threadIdx.x * V; i < end; i += THREADS * V) {
        float v[V];
        load_values<T, V>(p + i, v);
#pragma unroll
        for (int k = 0; k < V; ++k) part[k] = fmaf(v[k], v[k], part[k]);
    }
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) sum += part[k];
    const int i = (int)threadIdx.x < head ? threadIdx.x : end + (int)threadIdx.x - head;
    if (i < n) {
        const float v = static_cast<float>(p[i]);
        sum = fmaf(v, v, sum);
    }
    return sum;
}

// Where the result lies otherwise between 16-byte addresses than the gradient, one
// by one throughout.
template <int THREADS, typename T>
__device__ __forceinline__ void chunk_scale(const T *p, T *o, int n, float k) {
    constexpr int V = sizeof(T) == 4 ? 4 : 8;
    if ((reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(o)) % 16 == 0) {
        const int head = head_of(p, n), end = head + (n - head) / V * V;
#pragma unroll 4
        for (int i = head + threadIdx.x * V; i < end; i += THREADS * V) {
            float v[V];
            load_values<T, V>(p + i, v);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] *= k;
            store_values<T, V>(o + i, v);
        }
        const int i = (int)threadIdx.x < head ? threadIdx.x : end + (int)threadIdx.x - head;
        if (i < n) o[i] = static_cast<T>(static_cast<float>(p[i]) * k);
    } else {
#pragma unroll 8
        for (int i = threadIdx.x; i < n; i += THREADS) o[i] = static_cast<T>(static_cast<float>(p[i]) * k);
    }
}

// The squares of a chunk, and a chunk scaled, by its tensor's type.
template <int THREADS>
__device__ __forceinline__ float squares_of(const Tensor &t, int64_t at, int n) {
    if (t.type == GDN_DTYPE_F32) return chunk_squares<THREADS>(static_cast<const float *>(t.in) + at, n);
    if (t.type == GDN_DTYPE_F16) return chunk_squares<THREADS>(static_cast<const __half *>(t.in) + at, n);
    return chunk_squares<THREADS>(static_cast<const __nv_bfloat16 *>(t.in) + at, n);
}
template <int THREADS>
__device__ __forceinline__ void scale_to(const Tensor &t, int64_t at, int n, float k) {
    if (t.type == GDN_DTYPE_F32)
        chunk_scale<THREADS>(static_cast<const float *>(t.in) + at, static_cast<float *>(t.out) + at, n, k);
    else if (t.type == GDN_DTYPE_F16)
        chunk_scale<THREADS>(static_cast<const __half *>(t.in) + at, static_cast<__half *>(t.out) + at, n, k);
    else
        chunk_scale<THREADS>(static_cast<const __nv_bfloat16 *>(t.in) + at, static_cast<__nv_bfloat16 *>(t.out) + at, n,
                             k);
}
// The factor of a norm; 1 where it is not finite.
__device__ __forceinline__ float factor(float norm, float max_norm, float eps) {
    const float k = max_norm / (norm + eps);
    return isfinite(norm) && k < 1.f ? k : 1.f;
}
__device__ __forceinline__ void report(float norm, float *norm_out, int32_t *err) {
    if (norm_out) *norm_out = norm;
    if (!isfinite(norm) && err) atomicOr(err, kErrNonfinite);
}

template <int MAX>
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Table<MAX> tab, float *partial) {
    __shared__ float s[kThreads / 32];
    ptx::grid_wait();
    float sum = 0.f;
    for (int chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
        const Tensor &t = tab.t[find_tensor(tab, chunk)];
        const int64_t at = (int64_t)(chunk - t.first) * tab.chunk;
        const int n = (int)(t.n - at < tab.chunk ? t.n - at : tab.chunk);
        sum += squares_of<kThreads>(t, at, n);
    }
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) sum += s[w];
        partial[blockIdx.x] = sum;
    }
}

// Of partials that are not all finite: infinity or NaN, as their plain sum is.
__device__ __forceinline__ float plain_sum(const float *partial, int n) {
    float sum = 0.f;
    for (int i = 0; i < n; ++i) sum += partial[i];
    return sum;
}

template <int MAX>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<MAX> tab,
                                                        const float *partial, int partials, float max_norm, float eps,
                                                        float *norm_out, int32_t *err) {
    __shared__ TwoFloat s[kThreads / 32];
    ptx::grid_wait();
    TwoFloat sum = {0.f, 0.f};
    for (int i = threadIdx.x; i < partials; i += kThreads) sum = sum + TwoFloat{partial[i], 0.f};
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = s[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) sum = sum + s[w];
    // an infinite sum has a NaN beside it
    const float norm = sqrtf(isfinite(sum.hi + sum.lo) ? sum.hi + sum.lo : plain_sum(partial, partials));
    const float k = factor(norm, max_norm, eps);
    if (blockIdx.x == 0 && threadIdx.x == 0) report(norm, norm_out, err);
    for (int chunk = tab.chunks - 1 - (int)blockIdx.x; chunk >= 0; chunk -= (int)gridDim.x) {
        const Tensor &t = tab.t[find_tensor(tab, chunk)];
        if (k == 1.f && t.in == t.out) continue;
        const int64_t at = (int64_t)(chunk - t.first) * tab.chunk;
        const int n = (int)(t.n - at < tab.chunk ? t.n - at : tab.chunk);
        scale_to<kThreads>(t, at, n, k);
    }
}

// Fills a table with tensors i, i + 1, ...; returns the first that is not in it.
template <int MAX>
int fill(const gdn_grad_clip_args *a, int i, Table<MAX> *tab) {
    tab->count = tab->chunks = 0;
    int64_t elements = 0;
    for (int j = 0; j < a->count; ++j) elements += a->sizes[j];
    tab->chunk = elements <= kSmall ? kSmallChunk : kChunk;
    for (; i < a->count && tab->count < MAX; ++i) {
        if (a->sizes[i] == 0) continue;
        const int64_t chunks = (a->sizes[i] + tab->chunk - 1) / tab->chunk;
        if (tab->chunks + chunks > (1LL << 30)) break;
        Tensor &t = tab->t[tab->count++];
        t.in = a->grads[i];
        t.out = a->outs ? a->outs[i] : const_cast<void *>(a->grads[i]);
        t.n = a->sizes[i];
        t.first = tab->chunks;
        t.type = a->dtypes[i];
        tab->chunks += (int)chunks;
    }
    return i;
}

// Partials of all tables: one table's blocks after the other's.
template <int MAX>
int partial_count(const gdn_grad_clip_args *a) {
    Table<MAX> tab;
    int total = 0;
    for (int i = 0; i < a->count;) {
        i = fill<MAX>(a, i, &tab);
        total += tab.chunks < kBlocks ? tab.chunks : kBlocks;
    }
    return total;
}

template <int MAX>
cudaError_t run(const gdn_grad_clip_args *a, float *ws, cudaStream_t stream) {
    Table<MAX> tab;
    int total = 0;
    for (int i = 0; i < a->count;) {
        i = fill<MAX>(a, i, &tab);
        const int blocks = tab.chunks < kBlocks ? tab.chunks : kBlocks;
        if (blocks == 0) continue;
        const cudaError_t e = launch_early(squares_kernel<MAX>, blocks, kThreads, 0, stream, tab, ws + total);
        if (e != cudaSuccess) return e;
        total += blocks;
    }
    bool first = true;
    for (int i = 0; i < a->count || first; first = false) {
        i = fill<MAX>(a, i, &tab);
        const int blocks = tab.chunks < kBlocks ? tab.chunks : kBlocks;
        if (blocks == 0 && !first) continue;
        float *norm = first ? a->norm : nullptr;
        int32_t *err = first ? a->error_word : nullptr;
        const cudaError_t e = launch_early(scale_kernel<MAX>, blocks ? blocks : 1, kThreads, 0, stream, tab, ws, total,
                                           a->max_norm, a->eps, norm, err);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace clip
}  // namespace gdn

namespace {

using gdn::aligned;
using gdn::fail;

gdn_status validate(const gdn_grad_clip_args *a) {
    if (!a) return fail(GDN_ERR_INVALID, "args is NULL");
    if (a->count < 0) return fail(GDN_ERR_INVALID, "count must be >= 0");
    if (!(a->max_norm >= 0.f) || !isfinite(a->max_norm))
        return fail(GDN_ERR_INVALID, "max_norm must be >= 0 and finite");
    if (!(a->eps >= 0.f) || !isfinite(a->eps)) return fail(GDN_ERR_INVALID, "eps must be >= 0 and finite");
    if (a->count > 0 && (!a->grads || !a->sizes || !a->dtypes))
        return fail(GDN_ERR_INVALID, "grads, sizes and dtypes are required");
    for (int i = 0; i < a->count; ++i) {
        const int dt = a->dtypes[i];
        if (dt != GDN_DTYPE_F32 && dt != GDN_DTYPE_F16 && dt != GDN_DTYPE_BF16)
            return fail(GDN_ERR_INVALID, "tensor %d: unknown dtype %d", i, dt);
        if (a->sizes[i] < 0) return fail(GDN_ERR_INVALID, "tensor %d: size must be >= 0", i);
        if (a->sizes[i] > (1LL << 42)) return fail(GDN_ERR_UNSUPPORTED, "tensor %d: more than 2^42 elements", i);
        if (a->sizes[i] == 0) continue;
        const size_t e = dt == GDN_DTYPE_F32 ? 4 : 2;
        if (!a->grads[i] || (a->outs && !a->outs[i])) return fail(GDN_ERR_INVALID, "tensor %d: NULL", i);
        if (!aligned(a->grads[i], e) || (a->outs && !aligned(a->outs[i], e)))
            return fail(GDN_ERR_INVALID, "tensor %d is not aligned to its element size", i);
    }
    if (!aligned(a->norm, 4) || !aligned(a->error_word, 4))
        return fail(GDN_ERR_INVALID, "a pointer is not aligned to its element size");
    return GDN_OK;
}

// A table for few tensors keeps the launch's argument small.
constexpr int kFew = 32;
size_t workspace(const gdn_grad_clip_args *a) {
    const int n = a->count <= kFew ? gdn::clip::partial_count<kFew>(a) : gdn::clip::partial_count<gdn::clip::kMany>(a);
    return (size_t)(n + 3) / 4 * 16;
}

}  // namespace

extern "C" {

size_t gdn_grad_clip_workspace_size(const gdn_grad_clip_args *a) {
    if (validate(a) != GDN_OK) return (size_t)-1;
    gdn::ok();
    return workspace(a);
}

gdn_status gdn_grad_clip(const gdn_grad_clip_args *a, void *ws, size_t ws_bytes, gdn_stream stream) {
    const gdn_status st = validate(a);
    if (st != GDN_OK) return st;
    const size_t need = workspace(a);
    if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned(ws, 16)))
        return fail(GDN_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned (got %zu)", need, ws_bytes);
    float *w = static_cast<float *>(ws);
    cudaStream_t s = (cudaStream_t)stream;
    return gdn::cuda_status(a->count <= kFew ? gdn::clip::run<kFew>(a, w, s)
                                             : gdn::clip::run<gdn::clip::kMany>(a, w, s));
}

}  // extern "C"
