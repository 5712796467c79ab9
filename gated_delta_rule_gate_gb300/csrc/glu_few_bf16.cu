// glu_few_bf16.cu -- the gated feed-forward of few tokens and the element-wise parts of its gradient, bf16.
#include "glu_few.cuh"

namespace gdn {
namespace glu {
cudaError_t launch_few_bf16(const Few &p, cudaStream_t stream) { return launch_few<__nv_bfloat16>(p, stream); }
cudaError_t launch_gate_grad_bf16(const GateGrad &p, cudaStream_t stream) { return launch_gate_grad<__nv_bfloat16>(p, stream); }
cudaError_t launch_join_bf16(const Joins &p, cudaStream_t stream) { return launch_join<__nv_bfloat16>(p, stream); }
cudaError_t launch_forward_join_bf16(const ForwardJoin &p, cudaStream_t stream) {
    return launch_forward_join<__nv_bfloat16>(p, stream);
}
}  // namespace glu
}  // namespace gdn
