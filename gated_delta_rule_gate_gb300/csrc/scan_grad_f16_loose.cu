// scan_grad_f16_loose.cu -- gdn_scan_backward for f16 activations, rows anywhere.
#include "scan_bwd.cuh"

namespace gdn {
namespace scan {

cudaError_t launch_grad_f16_loose(const GradArgs &p, bool gate_f32, cudaStream_t stream) {
    return gate_f32 ? launch_grad_types<false, __half, float>(p, stream) : launch_grad_types<false, __half, __half>(p, stream);
}

}  // namespace scan
}  // namespace gdn
