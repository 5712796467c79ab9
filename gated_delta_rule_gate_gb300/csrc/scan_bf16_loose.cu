// scan_bf16_loose.cu -- gdn_scan for bf16 activations, rows anywhere.
#include "scan_fwd.cuh"

namespace gdn {
namespace scan {

cudaError_t launch_scan_bf16_loose(const Args &p, bool gate_f32, cudaStream_t stream) {
    return gate_f32 ? launch_types<false, __nv_bfloat16, float>(p, stream) : launch_types<false, __nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace scan
}  // namespace gdn
