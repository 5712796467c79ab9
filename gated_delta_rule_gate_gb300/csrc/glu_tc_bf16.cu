// glu_tc_bf16.cu -- the products of the gated feed-forward, bf16.
#include "glu_tc.cuh"

namespace gdn {
namespace glu {
cudaError_t launch_forward_bf16(const ForwardArgs &p, bool keep, cudaStream_t stream) {
    return launch_forward<__nv_bfloat16>(p, keep, stream);
}
cudaError_t launch_backward_bf16(const Backward &p, cudaStream_t stream) { return launch_product<__nv_bfloat16>(p, stream); }
}  // namespace glu
}  // namespace gdn
