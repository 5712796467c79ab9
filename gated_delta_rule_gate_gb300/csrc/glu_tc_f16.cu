// glu_tc_f16.cu -- the products of the gated feed-forward, fp16.
#include "glu_tc.cuh"

namespace gdn {
namespace glu {
cudaError_t launch_product_f16(const Product &p, Mode mode, cudaStream_t stream) {
    return launch_product<__half>(p, mode, stream);
}
}  // namespace glu
}  // namespace gdn
