// glu_launch.h -- what the host side of the gated feed-forward hands to its kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {
namespace glu {

// A result's rows: by tensor map where they are words of 16 bytes, else element by element.
struct Result {
    CUtensorMap map;
    void *at;
    int64_t stride;
    int by_map;
};
// One kind of product: results of the same sizes, each a sum over `pairs` pairs of operands
// (result z's are a[z + i], b[i] of pair i).  Tiles of 256 x 256, of 256 x 128 of the forward pass.
struct Job {
    CUtensorMap a[2], b[2];
    CUtensorMap shares;  // fp32 [parts x results (g and u of the forward pass), rows, cols], where parts > 1
    Result c[3];
    int64_t rows;
    uint32_t tiles;                 // of all results and stretches
    int cols, tiles_m, tiles_n, results;
    int pairs, blocks_k;            // K-steps (of 64) of one pair of operands
    int parts, per_part;            // stretches of K, and theirs
    int a_outer;                    // A has K as its outer dimension
};
// The forward pass: out = act(x w_gate^T) (x w_up^T); KEEP: the gates are results too;
// Shares: g and u of stretches of K are the results.
struct ForwardArgs {
    Job job;           // its results: out, and of kept gates the upper halves of g and u
    CUtensorMap lower; // and the next bytes of both
    int act;
    int32_t *err;
};
template <bool KEEP>
struct Forward : ForwardArgs {};
struct ForwardShares : ForwardArgs {};
// The gradients: dx = d_g w_gate + d_u w_up, and d_w = d^T x of both weights, in one launch.
struct Backward {
    Job job[2];
    int32_t *err;
};
// Fewer tokens than the tensor cores' tiles are made for.
struct Few {
    const void *x, *wg, *wu;
    void *out;
    unsigned char *gates;  // or null
    int64_t xs, os;
    int T, D, F, Fg, act, words;
};
// d_g and d_u of d_out and the gates that the forward pass kept.
struct GateGrad {
    const void *d_out;
    const unsigned char *gates;
    void *dg, *du;
    int64_t rows, dos;
    int F, Fp, Fg, act, words;  // Fp: elements between rows of dg and du; words: of d_out
};

// Kept gates: g and u cut to 24 bits.  A row is the upper 16 bits of g's Fg columns, those
// of u's, and then the next 8 bits, 64 columns of g and the same of u in turn.
constexpr int kGateColumns = 64;
__host__ __device__ constexpr int64_t gates_row(int Fg) { return 6 * (int64_t)Fg; }
__host__ __device__ constexpr int64_t lower_at(int Fg, int up, int col) {
    return 4 * (int64_t)Fg + col / kGateColumns * (2 * kGateColumns) + up * kGateColumns + col % kGateColumns;
}

// The shares of `parts` stretches added up and rounded: [parts, results, rows, cs] fp32.
struct Join {
    const float *shares;
    void *out[2];
    int64_t rows, stride;
    int cols, cs, parts, results, words;  // words: groups of four results are
};
struct Joins {
    Join j[2];
    int count;
};
// Those of the forward pass, [parts, g and u, rows, cs], joined before the activation.
struct ForwardJoin {
    const float *shares;
    void *out;
    unsigned char *gates;  // or null
    int64_t rows, os;
    int F, cs, Fg, parts, act, words;  // words: groups of four outputs are
};

// Up to so many tokens take the kernel of few.  32 tokens, fp16, weights that L2 does not hold, us:
// dim x inner            2048 x 1536  2048 x 2048  4096 x 1024  4096 x 4864  2048 x 6144  4096 x 8192
// this kernel                6.0          6.1          9.3          16.4         16.0         28.3
// the tensor cores' tiles   11.5         12.2         12.8          21.6         16.1         29.0
// (33 tokens in the tiles   11.7         12.5         13.1          21.8         16.2         29.1)
// So the border is where wide layers cross; narrow ones would gain from this kernel beyond it.
constexpr int kFewTokens = 32;

cudaError_t launch_forward_f16(const ForwardArgs &p, bool keep, cudaStream_t stream);
cudaError_t launch_forward_bf16(const ForwardArgs &p, bool keep, cudaStream_t stream);
cudaError_t launch_backward_f16(const Backward &p, cudaStream_t stream);
cudaError_t launch_backward_bf16(const Backward &p, cudaStream_t stream);
cudaError_t launch_few_f16(const Few &p, cudaStream_t stream);
cudaError_t launch_few_bf16(const Few &p, cudaStream_t stream);
cudaError_t launch_gate_grad_f16(const GateGrad &p, cudaStream_t stream);
cudaError_t launch_gate_grad_bf16(const GateGrad &p, cudaStream_t stream);
cudaError_t launch_join_f16(const Joins &p, cudaStream_t stream);
cudaError_t launch_join_bf16(const Joins &p, cudaStream_t stream);
cudaError_t launch_forward_join_f16(const ForwardJoin &p, cudaStream_t stream);
cudaError_t launch_forward_join_bf16(const ForwardJoin &p, cudaStream_t stream);

}  // namespace glu
}  // namespace gdn
