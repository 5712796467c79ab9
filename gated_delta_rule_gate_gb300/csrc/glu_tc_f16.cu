// glu_tc_f16.cu -- the products of the gated feed-forward, fp16.
#include "glu_tc.cuh"

namespace gdn {
namespace glu {
cudaError_t launch_forward_f16(const ForwardArgs &p, bool keep, cudaStream_t stream) {
    return launch_forward<__half>(p, keep, stream);
}
cudaError_t launch_backward_f16(const Backward &p, cudaStream_t stream) { return launch_product<__half>(p, stream); }
}  // namespace glu
}  // namespace gdn
