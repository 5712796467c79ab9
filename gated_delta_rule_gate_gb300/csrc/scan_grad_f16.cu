// scan_grad_f16.cu -- gdn_scan_backward for f16 activations, rows on 16-byte addresses.
#include "scan_bwd.cuh"

namespace gdn {
namespace scan {

cudaError_t launch_grad_f16(const GradArgs &p, bool gate_f32, cudaStream_t stream) {
    return gate_f32 ? launch_grad_types<true, __half, float>(p, stream) : launch_grad_types<true, __half, __half>(p, stream);
}

}  // namespace scan
}  // namespace gdn
