// rmsnorm_bf16.cu -- gdn_rmsnorm and its gradient for bf16 activations.
#include "rmsnorm.cuh"

namespace gdn {
namespace norm {

cudaError_t launch_bf16(const Args &p, int q, int width, cudaStream_t stream) {
    return launch_rmsnorm_as<__nv_bfloat16>(p, q, width, stream);
}

cudaError_t launch_grad_bf16(const GradArgs &p, bool r_f32, int width, int parts, float *ws, cudaStream_t stream) {
    return r_f32 ? launch_grad_as<__nv_bfloat16, float>(p, width, parts, ws, stream)
                 : launch_grad_as<__nv_bfloat16, __nv_bfloat16>(p, width, parts, ws, stream);
}

}  // namespace norm
}  // namespace gdn
