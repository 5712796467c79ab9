// scan_grad_bf16_loose.cu -- gdn_scan_backward for bf16 activations, rows anywhere.
#include "scan_bwd.cuh"

namespace gdn {
namespace scan {

cudaError_t launch_grad_bf16_loose(const GradArgs &p, bool gate_f32, cudaStream_t stream) {
    return gate_f32 ? launch_grad_types<false, __nv_bfloat16, float>(p, stream) : launch_grad_types<false, __nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace scan
}  // namespace gdn
