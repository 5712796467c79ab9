// rmsnorm_f32.cu -- gdn_rmsnorm and its gradient for f32 activations.
#include "rmsnorm.cuh"

namespace gdn {
namespace norm {

cudaError_t launch_f32(const Args &p, int q, bool vec, cudaStream_t stream) {
    return launch_rmsnorm_as<float>(p, q, vec, stream);
}

cudaError_t launch_grad_f32(const GradArgs &p, bool vec, int parts, float *ws, cudaStream_t stream) {
    return launch_grad_as<float, float>(p, vec, parts, ws, stream);
}

}  // namespace norm
}  // namespace gdn
