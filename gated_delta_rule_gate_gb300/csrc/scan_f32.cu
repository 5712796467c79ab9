// scan_f32.cu -- gdn_scan for f32 activations.
#include "scan_fwd.cuh"

namespace gdn {
namespace scan {

cudaError_t launch_scan_f32(const Args &p, cudaStream_t stream) {
    return launch_types<float, float>(p, stream);
}

}  // namespace scan
}  // namespace gdn
