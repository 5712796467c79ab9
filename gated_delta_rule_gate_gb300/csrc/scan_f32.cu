// scan_f32.cu -- gdn_scan for f32 activations, rows on 16-byte addresses.
#include "scan_fwd.cuh"

namespace gdn {
namespace scan {

cudaError_t launch_scan_f32(const Args &p, cudaStream_t stream) {
    return launch_types<true, float, float>(p, stream);
}

}  // namespace scan
}  // namespace gdn
