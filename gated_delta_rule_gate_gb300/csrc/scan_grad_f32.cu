// scan_grad_f32.cu -- gdn_scan_backward for f32 activations, rows on 16-byte addresses.
#include "scan_bwd.cuh"

namespace gdn {
namespace scan {

cudaError_t launch_grad_f32(const GradArgs &p, cudaStream_t stream) {
    return launch_grad_types<true, float, float>(p, stream);
}

}  // namespace scan
}  // namespace gdn
