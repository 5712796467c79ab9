// rmsnorm_launch.h -- host-side launchers of the norm (internal to libgdn).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {
namespace norm {

constexpr int kFit = 8192;   // values of a row that registers hold, at any alignment
constexpr int kNarrow = 32;  // longest rows that the gradient takes in pairs of fp32

struct Args {
    int64_t rows, xs;
    int D;
    float eps;
    int res_f32, w_f32;
    const void *x, *res, *weight;
    void *out, *res_out;
    float *scales, *rstd;
};
struct GradArgs {
    int64_t rows, dos;
    int D, Dp;  // Dp: D rounded up to whole words, the row of a block's share of d_weight
    int w_f32;
    const void *d_out, *r, *weight, *d_res;
    const float *rstd;
    void *dx;
    float *dw;
};

// q: 0 no scales, 1 a scale per row, 2 per group.  width: adjacent values that one
// word may take, everywhere: 8 (4 where a tensor of the row's is fp32), 2 or 1.
cudaError_t launch_f32(const Args &p, int q, int width, cudaStream_t stream);
cudaError_t launch_f16(const Args &p, int q, int width, cudaStream_t stream);
cudaError_t launch_bf16(const Args &p, int q, int width, cudaStream_t stream);
cudaError_t launch_grad_f32(const GradArgs &p, int width, int parts, float *ws, cudaStream_t stream);
cudaError_t launch_grad_f16(const GradArgs &p, bool r_f32, int width, int parts, float *ws, cudaStream_t stream);
cudaError_t launch_grad_bf16(const GradArgs &p, bool r_f32, int width, int parts, float *ws, cudaStream_t stream);
// d_weight = the sum of the blocks' shares.
cudaError_t launch_weight_sum(const float *partial, int parts, int D, int Dp, float *dw, cudaStream_t stream);

}  // namespace norm
}  // namespace gdn
