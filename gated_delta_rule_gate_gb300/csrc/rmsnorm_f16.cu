// rmsnorm_f16.cu -- gdn_rmsnorm and its gradient for f16 activations.
#include "rmsnorm.cuh"

namespace gdn {
namespace norm {

cudaError_t launch_f16(const Args &p, int q, int width, cudaStream_t stream) {
    return launch_rmsnorm_as<__half>(p, q, width, stream);
}

cudaError_t launch_grad_f16(const GradArgs &p, bool r_f32, int width, int parts, float *ws, cudaStream_t stream) {
    return r_f32 ? launch_grad_as<__half, float>(p, width, parts, ws, stream)
                 : launch_grad_as<__half, __half>(p, width, parts, ws, stream);
}

}  // namespace norm
}  // namespace gdn
