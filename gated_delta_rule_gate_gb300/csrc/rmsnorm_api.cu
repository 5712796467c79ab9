// rmsnorm_api.cu -- the C entry points of the norm: host-side validation and
// dispatch, and the sum of the blocks' shares of d_weight.
#include <math.h>

#include "launch.h"
#include "ptx.cuh"
#include "rmsnorm_launch.h"
#include "status.h"

namespace gdn {
namespace norm {

// 32 columns by 32 stretches of blocks a block; each column's sum in one order.
__global__ void __launch_bounds__(1024) weight_sum_kernel(const float *partial, int parts, int D, int Dp,
                                                          float *dw) {
    __shared__ float s[32][33];
    ptx::grid_wait();
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
    float sum = 0.f;
    if (c < D) {
#pragma unroll 8
        for (int b = k; b < parts; b += 32) sum += partial[(size_t)b * Dp + c];
    }
    s[k][threadIdx.x & 31] = sum;
    __syncthreads();
    if (k == 0 && c < D) {
        for (int i = 1; i < 32; ++i) sum += s[i][threadIdx.x];
        dw[c] = sum;
    }
}

cudaError_t launch_weight_sum(const float *partial, int parts, int D, int Dp, float *dw, cudaStream_t stream) {
    return launch_early(weight_sum_kernel, (unsigned)((D + 31) / 32), 1024, 0, stream, partial, parts, D, Dp, dw);
}

}  // namespace norm
}  // namespace gdn

namespace {

using gdn::aligned;
using gdn::fail;

constexpr int kMaxDim = 1 << 20;

size_t size_of(int dt) { return dt == GDN_DTYPE_F32 ? 4 : (dt == GDN_DTYPE_E4M3 ? 1 : 2); }
bool activation(int dt) { return dt == GDN_DTYPE_F32 || dt == GDN_DTYPE_F16 || dt == GDN_DTYPE_BF16; }
// Words of a row: 16 bytes of the narrowest tensor it is read with.
bool whole(const void *p, size_t e, int v) { return aligned(p, e * v < 16 ? e * v : 16); }

gdn_status check_common(int64_t rows, int dim, int x_dtype, int r_dtype, int w_dtype, int64_t stride,
                        const char *stride_name, const char *r_name) {
    if (rows < 0) return fail(GDN_ERR_INVALID, "rows must be >= 0");
    if (rows > (1LL << 31) - 1) return fail(GDN_ERR_UNSUPPORTED, "more than 2^31 - 1 rows are not supported");
    if (dim <= 0) return fail(GDN_ERR_INVALID, "dim must be positive (got %d)", dim);
    if (dim > kMaxDim) return fail(GDN_ERR_UNSUPPORTED, "dim above %d is not supported", kMaxDim);
    if (!activation(x_dtype)) return fail(GDN_ERR_INVALID, "x_dtype: unknown dtype %d", x_dtype);
    if (r_dtype != GDN_DTYPE_F32 && r_dtype != x_dtype)
        return fail(GDN_ERR_INVALID, "%s must be F32 or x_dtype", r_name);
    if (w_dtype != GDN_DTYPE_F32 && w_dtype != x_dtype)
        return fail(GDN_ERR_INVALID, "weight_dtype must be F32 or x_dtype");
    if (stride != 0 && stride < dim)
        return fail(GDN_ERR_INVALID, "%s (%lld) is less than dim (%d)", stride_name, (long long)stride, dim);
    return GDN_OK;
}

gdn_status validate_grad(const gdn_rmsnorm_grad_args *a) {
    if (!a) return fail(GDN_ERR_INVALID, "args is NULL");
    const gdn_status st = check_common(a->rows, a->dim, a->x_dtype, a->r_dtype, a->weight_dtype, a->d_out_stride,
                                       "d_out_stride", "r_dtype");
    if (st != GDN_OK) return st;
    if (!a->d_weight) return fail(GDN_ERR_INVALID, "d_weight is required");
    if (a->rows > 0 && (!a->d_out || !a->r || !a->weight || !a->rstd || !a->dx))
        return fail(GDN_ERR_INVALID, "d_out, r, weight, rstd and dx are required");
    const size_t ex = size_of(a->x_dtype), er = size_of(a->r_dtype);
    if (!aligned(a->d_out, ex) || !aligned(a->r, er) || !aligned(a->weight, size_of(a->weight_dtype)) ||
        !aligned(a->rstd, 4) || !aligned(a->d_residual, er) || !aligned(a->dx, er) || !aligned(a->d_weight, 4))
        return fail(GDN_ERR_INVALID, "a pointer is not aligned to its element size");
    return GDN_OK;
}

// Blocks that share the rows out: enough to fill the device at the row's size.  Four
// on each of 152 SMs: forward and gradient of 32768 x 2048 bf16 take 255, 206, 185,
// 202, 189 us with two, three, four, six, eight.
int grad_parts(const gdn_rmsnorm_grad_args *a) {
    if (a->rows == 0) return 0;
    int64_t n = 152 * 4;
    if (a->dim <= gdn::norm::kNarrow) n = 152 * 32;
    if (a->dim > gdn::norm::kFit) n = 152 * 4 / ((a->dim + 255) / 256) + 1;
    return (int)(a->rows < n ? a->rows : n);
}
int padded(int dim) { return (dim + 3) / 4 * 4; }
size_t grad_workspace(const gdn_rmsnorm_grad_args *a) {
    size_t n = (size_t)grad_parts(a) * padded(a->dim);
    if (a->dim > gdn::norm::kFit) n += (size_t)a->rows;
    return n * sizeof(float);
}

}  // namespace

extern "C" {

gdn_status gdn_rmsnorm(const gdn_rmsnorm_args *a, gdn_stream stream) {
    if (!a) return fail(GDN_ERR_INVALID, "args is NULL");
    const gdn_status st = check_common(a->rows, a->dim, a->x_dtype, a->residual ? a->residual_dtype : a->x_dtype,
                                       a->weight_dtype, a->x_stride, "x_stride", "residual_dtype");
    if (st != GDN_OK) return st;
    const bool quantised = a->out_dtype == GDN_DTYPE_E4M3;
    if (!quantised && a->out_dtype != a->x_dtype)
        return fail(GDN_ERR_INVALID, "out_dtype must be x_dtype or E4M3");
    if (a->group != 0 && !(quantised && a->group == 128))
        return fail(GDN_ERR_INVALID, "group must be 0, or 128 with an E4M3 output (got %d)", a->group);
    if (!(a->eps >= 0.f) || !isfinite(a->eps)) return fail(GDN_ERR_INVALID, "eps must be >= 0 and finite");
    if ((a->residual != nullptr) != (a->residual_out != nullptr) && a->rows > 0)
        return fail(GDN_ERR_INVALID, "residual and residual_out go together");
    if (quantised != (a->scales != nullptr) && a->rows > 0)
        return fail(GDN_ERR_INVALID, quantised ? "an E4M3 output needs scales" : "scales given without an E4M3 output");
    if (a->rows == 0) return gdn::ok();
    if (!a->x || !a->weight || !a->out) return fail(GDN_ERR_INVALID, "x, weight and out are required");
    const size_t ex = size_of(a->x_dtype), er = size_of(a->residual_dtype), ew = size_of(a->weight_dtype);
    if (!aligned(a->x, ex) || !aligned(a->residual, er) || !aligned(a->weight, ew) ||
        !aligned(a->out, size_of(a->out_dtype)) || !aligned(a->residual_out, er) || !aligned(a->scales, 4) ||
        !aligned(a->rstd, 4))
        return fail(GDN_ERR_INVALID, "a pointer is not aligned to its element size");
    gdn::norm::Args p;
    p.rows = a->rows;
    p.xs = a->x_stride ? a->x_stride : a->dim;
    p.D = a->dim;
    p.eps = a->eps;
    p.res_f32 = a->residual_dtype == GDN_DTYPE_F32;
    p.w_f32 = a->weight_dtype == GDN_DTYPE_F32;
    p.x = a->x, p.res = a->residual, p.weight = a->weight;
    p.out = a->out, p.res_out = a->residual_out, p.scales = a->scales, p.rstd = a->rstd;
    auto fits = [&](int v) {
        return p.D % v == 0 && p.xs % v == 0 && whole(a->x, ex, v) && whole(a->residual, er, v) &&
               whole(a->weight, ew, v) && whole(a->out, size_of(a->out_dtype), v) && whole(a->residual_out, er, v);
    };
    const int v = a->x_dtype == GDN_DTYPE_F32 ? 4 : 8, width = fits(v) ? v : fits(2) ? 2 : 1;
    const int q = !quantised ? 0 : (a->group ? 2 : 1);
    cudaStream_t s = (cudaStream_t)stream;
    if (a->x_dtype == GDN_DTYPE_F32) return gdn::cuda_status(gdn::norm::launch_f32(p, q, width, s));
    return gdn::cuda_status(a->x_dtype == GDN_DTYPE_F16 ? gdn::norm::launch_f16(p, q, width, s)
                                                        : gdn::norm::launch_bf16(p, q, width, s));
}

size_t gdn_rmsnorm_backward_workspace_size(const gdn_rmsnorm_grad_args *a) {
    if (validate_grad(a) != GDN_OK) return (size_t)-1;
    gdn::ok();
    return grad_workspace(a);
}

gdn_status gdn_rmsnorm_backward(const gdn_rmsnorm_grad_args *a, void *ws, size_t ws_bytes, gdn_stream stream) {
    const gdn_status st = validate_grad(a);
    if (st != GDN_OK) return st;
    const size_t need = grad_workspace(a);
    if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned(ws, 16)))
        return fail(GDN_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned (got %zu)", need, ws_bytes);
    cudaStream_t s = (cudaStream_t)stream;
    const int parts = grad_parts(a);
    float *w = static_cast<float *>(ws);
    if (parts > 0) {
        gdn::norm::GradArgs p;
        p.rows = a->rows;
        p.dos = a->d_out_stride ? a->d_out_stride : a->dim;
        p.D = a->dim;
        p.Dp = padded(a->dim);
        p.w_f32 = a->weight_dtype == GDN_DTYPE_F32;
        p.d_out = a->d_out, p.r = a->r, p.weight = a->weight, p.d_res = a->d_residual;
        p.rstd = a->rstd, p.dx = a->dx, p.dw = a->d_weight;
        const size_t ex = size_of(a->x_dtype), er = size_of(a->r_dtype), ew = size_of(a->weight_dtype);
        auto fits = [&](int v) {
            return p.D % v == 0 && p.dos % v == 0 && whole(a->d_out, ex, v) && whole(a->r, er, v) &&
                   whole(a->weight, ew, v) && whole(a->d_residual, er, v) && whole(a->dx, er, v);
        };
        const int v = a->r_dtype == GDN_DTYPE_F32 ? 4 : 8, width = fits(v) ? v : fits(2) ? 2 : 1;
        cudaError_t e;
        if (a->x_dtype == GDN_DTYPE_F32) e = gdn::norm::launch_grad_f32(p, width, parts, w, s);
        else if (a->x_dtype == GDN_DTYPE_F16)
            e = gdn::norm::launch_grad_f16(p, a->r_dtype == GDN_DTYPE_F32, width, parts, w, s);
        else e = gdn::norm::launch_grad_bf16(p, a->r_dtype == GDN_DTYPE_F32, width, parts, w, s);
        if (e != cudaSuccess) return gdn::cuda_status(e);
    }
    // without rows the sum is zero
    return gdn::cuda_status(gdn::norm::launch_weight_sum(w, parts, a->dim, padded(a->dim), a->d_weight, s));
}

}  // extern "C"
