// scan_grad_f32_loose.cu -- gdn_scan_backward for f32 activations, rows anywhere.
#include "scan_bwd.cuh"

namespace gdn {
namespace scan {

cudaError_t launch_grad_f32_loose(const GradArgs &p, cudaStream_t stream) {
    return launch_grad_types<false, float, float>(p, stream);
}

}  // namespace scan
}  // namespace gdn
