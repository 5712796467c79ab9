// scan_f16.cu -- gdn_scan for f16 activations, rows on 16-byte addresses.
#include "scan_fwd.cuh"

namespace gdn {
namespace scan {

cudaError_t launch_scan_f16(const Args &p, bool gate_f32, cudaStream_t stream) {
    return gate_f32 ? launch_types<true, __half, float>(p, stream) : launch_types<true, __half, __half>(p, stream);
}

}  // namespace scan
}  // namespace gdn
