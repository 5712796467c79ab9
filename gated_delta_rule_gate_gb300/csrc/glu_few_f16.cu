// glu_few_f16.cu -- the gated feed-forward of few tokens and the element-wise parts of its gradient, fp16.
#include "glu_few.cuh"

namespace gdn {
namespace glu {
cudaError_t launch_few_f16(const Few &p, cudaStream_t stream) { return launch_few<__half>(p, stream); }
cudaError_t launch_gate_grad_f16(const GateGrad &p, cudaStream_t stream) { return launch_gate_grad<__half>(p, stream); }
cudaError_t launch_join_f16(const Joins &p, cudaStream_t stream) { return launch_join<__half>(p, stream); }
cudaError_t launch_forward_join_f16(const ForwardJoin &p, cudaStream_t stream) {
    return launch_forward_join<__half>(p, stream);
}
}  // namespace glu
}  // namespace gdn
