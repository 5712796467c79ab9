// glu_tc_bf16.cu -- the products of the gated feed-forward, bf16.
#include "glu_tc.cuh"

namespace gdn {
namespace glu {
cudaError_t launch_product_bf16(const Product &p, Mode mode, cudaStream_t stream) {
    return launch_product<__nv_bfloat16>(p, mode, stream);
}
}  // namespace glu
}  // namespace gdn
