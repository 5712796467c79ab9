// glu_launch.h -- what the host side of the gated feed-forward hands to its kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {
namespace glu {

// The products, by the operands' order in memory and what is done with the result:
// kForward: out = act(x w_gate^T) (x w_up^T); kInput: dx = d_g w_gate + d_u w_up;
// kWeights: d_w = d^T x, of both weights.
enum Mode { kForward, kInput, kWeights };

// A result's rows: by tensor map where they are words of 16 bytes, else element by element.
struct Result {
    CUtensorMap map;
    void *at;
    int64_t stride;
    int by_map;
};
struct Product {
    CUtensorMap a[2], b[2];
    CUtensorMap shares;  // fp32 [parts x results, rows, cols], where parts > 1
    Result c[3];
    int64_t rows;
    uint32_t tiles;                  // of all results and stretches
    int cols, tiles_m, tiles_n;
    int blocks_k, parts, per_part;   // K-steps of one pair of operands; stretches of K, and theirs
    int act, gates;
    int32_t *err;
};
// Fewer tokens than the tensor cores' tiles are made for.
struct Few {
    const void *x, *wg, *wu;
    void *out, *gates;  // gates may be null
    int64_t xs, os;
    int T, D, F, Fp, act, words;
};
// d_g and d_u of d_out and the gates that the forward pass kept.
struct GateGrad {
    const void *d_out, *gates;
    void *dg, *du;
    int64_t rows, dos;
    int F, Fp, act, words;  // Fp: elements between g and u, and between rows of dg and du; words: of d_out
};

// The shares of `parts` stretches added up and rounded: [parts, results, rows, cs] fp32.
struct Join {
    const float *shares;
    void *out[2];
    int64_t rows, stride;
    int cols, cs, parts, results;
};

constexpr int kFewTokens = 16;

cudaError_t launch_product_f16(const Product &p, Mode mode, cudaStream_t stream);
cudaError_t launch_product_bf16(const Product &p, Mode mode, cudaStream_t stream);
cudaError_t launch_few_f16(const Few &p, cudaStream_t stream);
cudaError_t launch_few_bf16(const Few &p, cudaStream_t stream);
cudaError_t launch_gate_grad_f16(const GateGrad &p, cudaStream_t stream);
cudaError_t launch_gate_grad_bf16(const GateGrad &p, cudaStream_t stream);
cudaError_t launch_join_f16(const Join &p, cudaStream_t stream);
cudaError_t launch_join_bf16(const Join &p, cudaStream_t stream);

}  // namespace glu
}  // namespace gdn
