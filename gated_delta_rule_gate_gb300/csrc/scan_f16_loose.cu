// scan_f16_loose.cu -- gdn_scan for f16 activations, rows anywhere.
#include "scan_fwd.cuh"

namespace gdn {
namespace scan {

cudaError_t launch_scan_f16_loose(const Args &p, bool gate_f32, cudaStream_t stream) {
    return gate_f32 ? launch_types<false, __half, float>(p, stream) : launch_types<false, __half, __half>(p, stream);
}

}  // namespace scan
}  // namespace gdn
