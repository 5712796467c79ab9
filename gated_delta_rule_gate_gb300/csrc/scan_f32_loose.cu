// scan_f32_loose.cu -- gdn_scan for f32 activations, rows anywhere.
#include "scan_fwd.cuh"

namespace gdn {
namespace scan {

cudaError_t launch_scan_f32_loose(const Args &p, cudaStream_t stream) {
    return launch_types<false, float, float>(p, stream);
}

}  // namespace scan
}  // namespace gdn
