// scan_step.cu -- gdn_scan_step: the gated linear recurrence, the tokens of a
// request one after another (one or a few tokens a request).
//
// A thread holds the states of V adjacent channels of one request in registers
// and walks its tokens: h = a h + n i x.  Bound by HBM at many requests (a state
// row in and out, 8 bytes a channel, beside the token's tensors) and by launch
// and memory latency at few; all loads of a token are issued together.  256 x 4096
// fp16 with raw and input gates 4.4 us, of which HBM takes 2.5; 1 x 2048 3.1 us.
#include "launch.h"
#include "ptx.cuh"
#include "scan_launch.h"

namespace gdn {
namespace scan {

template <typename T, int V>
__device__ __forceinline__ void load_channels(const T *p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = static_cast<float>(*p);
    } else if constexpr (sizeof(T) == 4) {
        const float4 r = *reinterpret_cast<const float4 *>(p);
        v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
    } else {
        const uint2 r = *reinterpret_cast<const uint2 *>(p);
        const float2 a = unpack<T>(r.x), b = unpack<T>(r.y);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_channels(T *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = static_cast<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(pack<T>(make_float2(v[0], v[1])), pack<T>(make_float2(v[2], v[3])));
    }
}

constexpr int kThreads = 128;

template <typename TA, typename TG, int V>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(const __grid_constant__ Args p, int blocks) {
    ptx::grid_wait();
    const int b = blockIdx.x / blocks;
    const int c = ((blockIdx.x % blocks) * kThreads + threadIdx.x) * V;
    int t0, t1;
    request_tokens(p, b, t0, t1);
    const int row = request_row(p, b);
    if (threadIdx.x == 0 && blockIdx.x % blocks == 0 && p.err) {
        if (row < 0) atomicOr(p.err, kErrBadSlot);
        if (p.cu && clamped_offset(p, b + 1) < clamped_offset(p, b)) atomicOr(p.err, kErrOverlap);
    }
    if (row < 0 || c >= p.D) return;
    float h[V] = {};
    const size_t at = (size_t)row * p.D + c;
    if (p.init) load_channels<float, V>(p.init + at, h);
    float bias[V] = {}, scale[V] = {};
    if (p.bias) {
        load_channels<float, V>(p.bias + c, bias);
        load_channels<float, V>(p.scale + c, scale);
    }
    for (int t = t0; t < t1; ++t) {
        float x[V], z[V], y[V] = {};
        load_channels<TA, V>(static_cast<const TA *>(p.x) + t * p.xs + c, x);
        load_channels<TG, V>(static_cast<const TG *>(p.decay) + t * p.gs + c, z);
        if (p.beta) load_channels<TG, V>(static_cast<const TG *>(p.beta) + t * p.bs + c, y);
        constexpr int W = V > 1 ? V / 2 : 1;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int i = 2 * w, j = V > 1 ? i + 1 : i;
            const float2 zz = make_float2(z[i], z[j]), yy = make_float2(y[i], y[j]);
            const float2 bb = make_float2(bias[i], bias[j]), ss = make_float2(scale[i], scale[j]);
            const Exp e = exponential(p.bias ? log_decay<true>(zz, bb, ss) : zz);
            float2 u = make_float2(x[i], x[j]);
            if (p.beta) u = u * (p.sigmoid ? sigmoid(yy) : yy);
            if (p.mode == kLerp) u = u * -e.m;
            if (p.mode == kUnit) u = u * unit_scale(e.m);
            const float2 r = fma2(e.a, make_float2(h[i], h[j]), u);
            h[i] = r.x;
            h[j] = V > 1 ? r.y : r.x;
        }
        store_channels<TA, V>(static_cast<TA *>(p.o) + t * p.os + c, h);
    }
    if (p.fin && (t1 > t0 || p.fin != p.init)) store_channels<float, V>(p.fin + at, h);
}

template <typename TA, typename TG>
static cudaError_t launch(const Args &p, bool vec4, cudaStream_t stream) {
    const int per = kThreads * (vec4 ? 4 : 1);
    const int blocks = (p.D + per - 1) / per;
    const unsigned grid = (unsigned)blocks * (unsigned)p.B;
    return launch_early(vec4 ? scan_step_kernel<TA, TG, 4> : scan_step_kernel<TA, TG, 1>, grid, kThreads, 0, stream, p,
                        blocks);
}

cudaError_t launch_step(const Args &p, int act, int gate, bool vec4, cudaStream_t stream) {
    if (act == 0) return launch<float, float>(p, vec4, stream);
    if (act == 1)
        return gate ? launch<__half, __half>(p, vec4, stream) : launch<__half, float>(p, vec4, stream);
    return gate ? launch<__nv_bfloat16, __nv_bfloat16>(p, vec4, stream)
                : launch<__nv_bfloat16, float>(p, vec4, stream);
}

}  // namespace scan
}  // namespace gdn
