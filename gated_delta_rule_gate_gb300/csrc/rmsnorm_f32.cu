// rmsnorm_f32.cu -- gdn_rmsnorm and its gradient for f32 activations.
#include "rmsnorm.cuh"

namespace gdn {
namespace norm {

cudaError_t launch_f32(const Args &p, int q, int width, cudaStream_t stream) {
    return launch_rmsnorm_as<float>(p, q, width, stream);
}

cudaError_t launch_grad_f32(const GradArgs &p, int width, int parts, float *ws, cudaStream_t stream) {
    return launch_grad_as<float, float>(p, width, parts, ws, stream);
}

}  // namespace norm
}  // namespace gdn
