/*
 * gdn.h -- C ABI of the gated delta rule library (libgdn.so, sm_103a).
 *
 * The operation (value-major storage; S is dv x dk fp32 per value head):
 *
 *   per token t of a request, for each value head h (query/key head
 *   qh = h * Hq / Hv):
 *     alpha = exp(g_t)                      (scalar, or a dk-vector per key)
 *     S     = S * Diag(alpha)               (decay; rules gated, gated_delta, gdn2)
 *     u     = S kappa                       (retrieval; rules delta, gated_delta, gdn2)
 *     d     = beta_t (v_t - u)              (delta, gated_delta)
 *     d     = beta_t (w_t .* v_t) - u       (gdn2; kappa = b_t .* k_t; beta_t = 1
 *                                            when the erase gate rides in beta,
 *                                            w_t = 1 without a write gate)
 *     d     = v_t                           (linear, gated)
 *     S     = S + d k_t^T
 *     o_t   = scale * S q_t
 *
 * Sources: "com.microsoft.GatedDeltaNet" README (Description, Inputs,
 * Outputs, Attributes); "com.microsoft.LinearAttentionGate" (Description);
 * "aclnnRecurrentGatedDeltaRule" (Formula; two-phase workspace query);
 * "gatedDeltaUpdate" (CLIKA runtime: slot_ids slab, raw-gate arm, per-key
 * gate, key-major state slab); ONNX issue "Spec gap: LinearAttention
 * (opset 27) cannot represent Gated DeltaNet-2 channel-wise erase gate"
 * (proposals A and B, and the write gate of its first display).
 *
 * Conventions for every entry point:
 *  - Every tensor pointer is DEVICE memory owned by the caller, row-major and
 *    contiguous in the layout stated, aligned at least to its element size.
 *    The library allocates no device memory and keeps no pointer after the
 *    call returns.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default
 *    stream) and runs asynchronously: no entry point synchronises.  Inputs
 *    must stay valid and outputs must not be read until the stream reaches
 *    the work.
 *  - Arguments are validated on the host before anything is launched; a
 *    non-OK status means nothing was enqueued and no output was touched.
 *    gdn_last_error_message() then describes the first failed check.
 *  - All entry points are thread-safe (the message is thread-local).
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t, declared without the CUDA headers. */
typedef struct CUstream_st *gdn_stream;

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_ERR_INVALID = 1,     /* the arguments break the op contract */
    GDN_ERR_UNSUPPORTED = 2, /* a valid request this library declines (typed) */
    GDN_ERR_WORKSPACE = 3,   /* workspace missing, too small or misaligned */
    GDN_ERR_CUDA = 4         /* a CUDA launch or runtime call failed */
} gdn_status;

typedef enum gdn_dtype {
    GDN_DTYPE_F32 = 0,
    GDN_DTYPE_F16 = 1,
    GDN_DTYPE_BF16 = 2, /* the recurrent-layer operators; the others decline it: GDN_ERR_UNSUPPORTED */
    GDN_DTYPE_E4M3 = 3  /* 8 bits (4 of exponent, 3 of mantissa, largest 448): output of gdn_rmsnorm, states of gdn_adamw */
} gdn_dtype;

/* "com.microsoft.GatedDeltaNet", Attributes, update_rule; GDN2 is the rule
 * of the ONNX "Spec gap ... Gated DeltaNet-2" issue (its erase gate in beta,
 * proposal A, or in erase_gate, proposal B). */
typedef enum gdn_rule {
    GDN_RULE_LINEAR = 0,      /* no decay, no retrieval: S += v k^T */
    GDN_RULE_GATED = 1,       /* decay only */
    GDN_RULE_DELTA = 2,       /* retrieval only */
    GDN_RULE_GATED_DELTA = 3, /* both (the default of the op) */
    GDN_RULE_GDN2 = 4         /* decay, then erase with kappa = b .* k, write k v^T */
} gdn_rule;

/* Flags (gdn_problem.flags). */
#define GDN_FLAG_L2NORM_Q 0x1u      /* q <- q / sqrt(sum q^2 + 1e-12) first (qk_l2_norm) */
#define GDN_FLAG_L2NORM_K 0x2u      /* same for k */
#define GDN_FLAG_BETA_SIGMOID 0x4u  /* beta <- sigmoid(beta) in fp32 (beta_activation) */
#define GDN_FLAG_DECAY_PER_KEY 0x8u /* decay is [.., Hv, dk]: one log-decay per key channel */
#define GDN_FLAG_BETA_SHARED 0x10u  /* beta is [total_tokens]: one per token, shared by every value head */
#define GDN_FLAG_STATE_KMAJOR 0x20u /* states are key-major [num_state_rows, Hv, dk, dv] ("gatedDeltaUpdate") */

/* Bits OR-ed into *error_word by the device (never reset by the library). */
#define GDN_DEVERR_BAD_SLOT 0x1 /* a slot id outside [0, num_state_rows): request skipped */
#define GDN_DEVERR_TIMEOUT 0x2  /* a bounded wait on an asynchronous copy ran out: the CTA gave up */
#define GDN_DEVERR_OVERLAP 0x4  /* chunked prefill: the requests' chunks outgrew the workspace, which only
                                   requests sharing tokens can do; the requests past it were skipped */
#define GDN_DEVERR_DECAY_RANGE 0x8 /* chunked prefill, per-key decay on the tensor cores: a log decay above 0
                                      (a decay above 1) was given; that path needs decays in (0, 1] and the
                                      results of the chunks concerned are not valid */

#define GDN_DEVERR_NONFINITE 0x10 /* gdn_grad_clip: the norm is infinite or NaN; the gradients were not scaled.
                                     gdn_adamw: grad_norm is; the step was not taken */

/*
 * One call of the recurrence over a batch of requests.
 *
 * Token layout.  Rank-3 packed form (seq_len == 0): q, k are
 * [total_tokens, Hq, dk], v and o are [total_tokens, Hv, dv].  Request b owns
 * tokens [clamp(cu_seqlens[b]), clamp(cu_seqlens[b+1])), each clamped to
 * [0, total_tokens]; a decreasing pair gives an empty request (GatedDeltaNet
 * Inputs table, cu_seqlens).  cu_seqlens NULL means uniform packing:
 * total_tokens / batch tokens each (total_tokens must divide).  Output tokens
 * that no request covers are not written.
 * Rank-4 form (seq_len > 0): q, k are [batch, seq_len, Hq, dk] (the same
 * memory layout), total_tokens must equal batch * seq_len, and cu_seqlens must
 * be NULL (the op allows cu_seqlens with the rank-3 spelling only).  seq_lens
 * (rank-4 form only; "gatedDeltaUpdate", seq_lens bounds the rows of a ragged
 * prefill) makes the batch padded-ragged: request b owns the first
 * clamp(seq_lens[b], 0, seq_len) tokens of its row, [b * seq_len,
 * b * seq_len + that); the padding tokens take no part in any result and
 * are not written (their contents may be anything, NaN included).
 * seq_lens NULL means every row is full.
 *
 * Heads.  num_heads_v is a positive multiple of num_heads_q; value head h
 * reads query/key head h * Hq / Hv.
 *
 * Gate (decay).  Present exactly for rules GATED, GATED_DELTA and GDN2.
 *  - gate_bias == gate_scale == NULL: `decay` is the log-space decay g.
 *  - both non-NULL (raw-gate arm, gatedDeltaUpdate): `decay` is the raw gate
 *    projection and g = gate_scale[h] * softplus(decay + gate_bias) is formed
 *    in fp32 inside the kernel.  gate_bias is [Hv] (or [Hv, dk] with
 *    GDN_FLAG_DECAY_PER_KEY), gate_scale is [Hv] (the folded -exp(A_log)).
 *  - exactly one of them non-NULL: GDN_ERR_INVALID.
 *  decay is [total_tokens, Hv], or [total_tokens, Hv, dk] with
 *  GDN_FLAG_DECAY_PER_KEY; decay_dtype is F32 or act_dtype.
 *
 * Beta.  Present exactly for rules DELTA, GATED_DELTA (shape [total_tokens,
 * Hv], or [total_tokens] with GDN_FLAG_BETA_SHARED: beta's last dimension 1,
 * broadcast over the value heads, as the LinearAttention schema allows) and
 * GDN2 (the erase gate b, [total_tokens, Hv, dk], when erase_gate is NULL;
 * GDN_FLAG_BETA_SHARED is then rejected); beta_dtype is F32 or act_dtype;
 * GDN_FLAG_BETA_SIGMOID applies the logistic sigmoid first.
 *
 * GDN2 gates (ONNX GDN-2 issue).  erase_gate (proposal B) is the erase gate b
 * as an input of its own, fp32 [total_tokens, Hv, dk], taken as given (no
 * activation); beta is then the scalar write rate of DELTA / GATED_DELTA
 * ([total_tokens, Hv], or [total_tokens] with GDN_FLAG_BETA_SHARED; the
 * sigmoid flag applies to it), so erase_gate = beta * 1 gives GATED_DELTA.
 * write_gate is the write gate w, fp32 [total_tokens, Hv, dv], multiplied
 * into v inside the kernels (NULL: w = 1, or already folded into v by the
 * caller).  Both are GDN2 only (GDN_ERR_INVALID otherwise).
 *
 * State.  initial_state and final_state are fp32, value-major
 * [num_state_rows, Hv, dv, dk], or key-major [num_state_rows, Hv, dk, dv]
 * with GDN_FLAG_STATE_KMAJOR (the slab layout of "gatedDeltaUpdate"; the
 * recurrence is the same).  Request b reads and writes row
 * slot_ids[b] if slot_ids is non-NULL (the slab of gatedDeltaUpdate), else
 * row b.  initial_state NULL means a zero state.  final_state may equal
 * initial_state (in-place update); otherwise the two must not overlap.  Rows
 * no request names are not touched.  An empty request leaves its final
 * state equal to its initial state ("com.microsoft.GatedDeltaNet",
 * Outputs).  Slot ids must be distinct (caller's contract); a slot id outside [0, num_state_rows) makes every CTA of that request skip it
 * and OR GDN_DEVERR_BAD_SLOT into *error_word (if error_word is non-NULL).
 *
 * scale == 0 selects 1/sqrt(dk).  state_update_capacity must be 0 (compact
 * transition capture is not part of this library).
 */
typedef struct gdn_problem {
    int32_t batch;          /* B: number of requests (0: nothing to do) */
    int32_t total_tokens;   /* T */
    int32_t seq_len;        /* 0: rank-3 packed; > 0: rank-4 uniform */
    int32_t num_heads_q;    /* Hq */
    int32_t num_heads_v;    /* Hv */
    int32_t head_dim_k;     /* dk */
    int32_t head_dim_v;     /* dv */
    int32_t num_state_rows; /* rows of the state tensors; 0 means batch */
    int32_t act_dtype;      /* gdn_dtype of q, k, v, o: F32 or F16 */
    int32_t decay_dtype;    /* gdn_dtype of decay: F32 or act_dtype */
    int32_t beta_dtype;     /* gdn_dtype of beta: F32 or act_dtype */
    int32_t rule;           /* gdn_rule */
    uint32_t flags;         /* GDN_FLAG_* */
    float scale;            /* 0: 1/sqrt(dk) */
    int32_t state_update_capacity; /* must be 0 */
    const void *q;
    const void *k;
    const void *v;
    void *o;
    const void *decay;
    const float *gate_bias;
    const float *gate_scale;
    const void *beta;
    const int32_t *cu_seqlens; /* [batch + 1] or NULL */
    const int32_t *slot_ids;   /* [batch] or NULL */
    const float *initial_state;
    float *final_state;
    int32_t *error_word; /* optional device int32 */
    const int32_t *seq_lens; /* [batch] or NULL: rank-4 form only (see Token layout) */
    const float *erase_gate; /* GDN2 only: [total_tokens, Hv, dk] fp32, or NULL (see GDN2 gates) */
    const float *write_gate; /* GDN2 only: [total_tokens, Hv, dv] fp32, or NULL (see GDN2 gates) */
} gdn_problem;

/*
 * gdn_gate -- "com.microsoft.LinearAttentionGate", Description:
 *   decay = decay_scale * softplus(a + dt_bias)   and, if beta_out != NULL,
 *   beta  = sigmoid(b).
 * a (and b) are [n, heads]: any leading axes folded into n, heads last.
 * dt_bias and decay_scale are fp32 [heads].  a, b, decay_out and beta_out
 * share `dtype` (F32 or F16).  Arithmetic is fp32, rounded once on store.
 * beta_out requires b (GDN_ERR_INVALID otherwise); b without beta_out is
 * accepted and unused.  n == 0 is a no-op.
 */
typedef struct gdn_gate_args {
    int64_t n;
    int32_t heads;
    int32_t dtype;
    const void *a;
    const float *dt_bias;
    const float *decay_scale;
    const void *b;
    void *decay_out;
    void *beta_out;
} gdn_gate_args;

gdn_status gdn_gate(const gdn_gate_args *args, gdn_stream stream);

/*
 * gdn_recurrent_step -- token-serial recurrence ("aclnnRecurrentGatedDeltaRule":
 * the variable-step-size form, designed for L_i <= 8 tokens per request, the
 * decode / multi-token-prediction step).  Any request length is accepted;
 * time grows linearly with the longest request.  Supports every rule, both
 * gate arms, per-key decay, GDN2, 1 <= dk, dv <= 256 (larger:
 * GDN_ERR_UNSUPPORTED).  fp32 arithmetic throughout; the state tile of each
 * (request, value head) crosses HBM once each way.
 */
gdn_status gdn_recurrent_step(const gdn_problem *p, gdn_stream stream);

/*
 * gdn_chunked_prefill_workspace_size -- bytes of device workspace that
 * gdn_chunked_prefill needs for this problem and chunk size (the first phase
 * of the two-phase style of "aclnnRecurrentGatedDeltaRule").  Returns 0 when
 * no workspace is needed, and (size_t)-1 when the problem is rejected (the
 * reason is then in gdn_last_error_message()).
 */
size_t gdn_chunked_prefill_workspace_size(const gdn_problem *p, int32_t chunk_size);

/*
 * gdn_chunked_prefill_workspace_size_min -- the least workspace
 * gdn_chunked_prefill accepts for this problem (0, (size_t)-1 as above).  It
 * holds one chunk of every request at a time, so it does not grow with the
 * request lengths (the fp32-activation and fp16-gate copies aside).  With any
 * workspace from this size up to gdn_chunked_prefill_workspace_size() the call
 * runs in windows of as many chunks per request as fit, one after another on
 * the stream: each window reads the state the previous one left in
 * final_state (fp32, so the result is the same, bit for bit, as a single pass)
 * and writes its tokens' outputs.  Not an operation of the pages: a bound on
 * the library's own scratch ("aclnnRecurrentGatedDeltaRule" asks for its
 * workspace in a first phase; this is the least of it).
 */
size_t gdn_chunked_prefill_workspace_size_min(const gdn_problem *p, int32_t chunk_size);

/*
 * gdn_chunked_prefill -- the same result as gdn_recurrent_step, computed
 * chunk-parallel: within a chunk the delta rule becomes a unit-lower-
 * triangular system solved once per chunk, and the intra-chunk attention and
 * the state carry-in/carry-out become dense fp16 tensor-core products with
 * fp32 accumulation; the state itself stays fp32 across chunks.
 * ("com.microsoft.GatedDeltaNet", Attributes, chunk_size: any value is
 * accepted and none changes the result beyond rounding; <= 0 selects 64.)
 * Extra constraints (GDN_ERR_UNSUPPORTED otherwise): dk in {16, 32, 64, 128},
 * dv a multiple of 16 (<= 256), q, k, v, o and the state 16-byte aligned.
 * fp32 activations are rounded to fp16 for the products (at dk = dv = 128
 * through fp16 copies of q, k and v that the library writes into the
 * workspace; o is still written in fp32).  Per-key decay (gated, gated_delta)
 * and GDN2 run on the tensor cores when dk = dv = 128 and the per-key gate
 * rows are 16-byte aligned (fp16 per-key log decays, and GDN2's fp16 per-key
 * beta, through fp32 copies that the library writes into the workspace);
 * per-key log decays are expected <= 0 there (decays in (0, 1], as the
 * raw-gate arm always gives).  Per-key problems at other head sizes run the
 * token-serial form (same result).
 *
 * Workspace: owned by the caller, device memory of at least
 * gdn_chunked_prefill_workspace_size_min() bytes, 256-byte aligned (NULL
 * allowed when that is 0); GDN_ERR_WORKSPACE otherwise.  Below
 * gdn_chunked_prefill_workspace_size() the call runs in windows (see
 * gdn_chunked_prefill_workspace_size_min).  It is non-zero whenever the
 * tensor-core path runs (every rule with dk = dv = 128, per-key problems as
 * above), and 0 otherwise.  Layout, for T / 64 + B + 1 chunk slots:
 * per-request chunk offsets, a chunk-slot -> request table and the requests
 * ordered by length (rounded up to 1 KB); then one 88 KB image per (chunk
 * slot, value head) of the chunk's state-independent operands (fp16); with
 * fp32 activations, the fp16 copies of q, k and v (each rounded up to 256
 * bytes); last, fp32 copies [total_tokens, Hv, 128] of fp16 per-key gate rows
 * (the log decay; GDN2's per-key beta), each rounded up to 256 bytes.
 * Its contents are scratch, rewritten by every call on the stream; two calls
 * in flight at once need two workspaces.  Requests that share tokens can need
 * more slots than that; the ones past the capacity are skipped and
 * GDN_DEVERR_OVERLAP is set.
 */
gdn_status gdn_chunked_prefill(const gdn_problem *p, int32_t chunk_size, void *workspace,
                               size_t workspace_bytes, gdn_stream stream);

/*
 * gdn_chunked_prefill_noalloc -- gdn_chunked_prefill with the library's own
 * scratch instead of a caller workspace.  None of the reference pages has a
 * counterpart of this entry point; it exists for callers that cannot allocate
 * device memory around the call.
 *
 * The scratch is one static device array of 768 MiB per device (set aside
 * when libgdn loads; this entry point allocates nothing).  Each process that
 * loads libgdn reserves its own 768 MiB on every device it uses, so calls
 * from different processes never share it.  Problems whose
 * gdn_chunked_prefill_workspace_size() exceeds it are rejected on the host
 * with GDN_ERR_WORKSPACE before anything is enqueued (the long and ragged
 * prefill configurations, about 745-765 MB, fit).  Within a process, every
 * call on a device shares the array: two calls in flight at the same time on
 * that device (different streams or threads) race on it, so the caller
 * serialises them.  Every call looks the array's address up on the current
 * device (cudaGetSymbolAddress), so the address stays right after a device
 * reset; the first call on each device also sets kernel attributes: make it
 * outside any stream capture.  Same arguments, constraints, results and
 * error bits as gdn_chunked_prefill.
 */
gdn_status gdn_chunked_prefill_noalloc(const gdn_problem *p, int32_t chunk_size, gdn_stream stream);

/*
 * Recurrent-layer operators: what a layer runs around and instead of the
 * matrix-state recurrence -- a gated linear recurrence of vector state with its
 * gradient, the norm at the layer's entry, the clipping of the gradients.  The
 * reference pages define none of them (the gate's raw arm is theirs).  They
 * take F32, F16 and BF16 tensors.
 */

/* Scale n of a token's input in gdn_scan. */
typedef enum gdn_input_scale {
    GDN_INPUT_SCALE_NONE = 0, /* n = 1 */
    GDN_INPUT_SCALE_LERP = 1, /* n = 1 - a: the state is a running mean */
    GDN_INPUT_SCALE_UNIT = 2  /* n = sqrt(1 - a^2): unit-variance inputs keep the state at unit variance */
} gdn_input_scale;

/* Tokens between two entries of gdn_scan's chunk_states. */
#define GDN_SCAN_CHUNK 64

/*
 * One call of the gated linear recurrence, per token t and channel c:
 *
 *     g   = decay                                  (gate_bias == gate_scale == NULL)
 *     g   = gate_scale[c] * softplus(decay + gate_bias[c])   (both given: the raw arm)
 *     a   = exp(g)
 *     i   = 1 | beta | sigmoid(beta)               (beta NULL | given | GDN_FLAG_BETA_SIGMOID)
 *     n   = 1 | 1 - a | sqrt(max(0, 1 - a^2))      (input_scale)
 *     h_t = a h_{t-1} + n i x_t,   o_t = h_t
 *
 * The state h is fp32; o is rounded once.  a is good to (4 + 1.25 |g|) 2^-24 of itself,
 * and 0 where it is below 2^-126.  g <= 0 is expected (g = -inf forgets
 * the past; g > 0 grows the state and makes n <= 0 with LERP and 0 with UNIT).  Runs of
 * tokens may grow or shrink by more than fp32 holds; a state that is a number
 * after every token comes out as one.
 *
 * Tokens and requests are those of gdn_problem: seq_len == 0 is the packed form
 * ([total_tokens, channels]; request b owns tokens [cu_seqlens[b],
 * cu_seqlens[b + 1]), each clamped to [0, total_tokens]; cu_seqlens NULL: batch
 * requests of total_tokens / batch), seq_len > 0 the uniform form ([batch,
 * seq_len, channels]), which seq_lens makes padded.  Here the clamped offsets
 * must not decrease (equal ones: an empty request); a decreasing pair sets
 * GDN_DEVERR_OVERLAP and the results of that call are unspecified (in bounds).
 * Tokens of no request take no part in any result and are not written.
 *
 * x, decay, beta and o have channels contiguous and *_stride elements from one
 * token to the next (0: channels), so that they may be columns of a wider
 * matrix; a stride must be at least channels.  o overlaps no input.
 *
 * States are [num_state_rows, channels] fp32, rows by slot_ids or by request, as
 * in gdn_problem: initial_state NULL is zero; final_state may be NULL, may equal
 * initial_state, and receives an empty request's initial state.  A bad slot id
 * skips the request and sets GDN_DEVERR_BAD_SLOT.
 *
 * chunk_states (gdn_scan only; NULL: not kept) is fp32
 * [ceil(total_tokens / GDN_SCAN_CHUNK), channels]: entry j receives the state
 * before token j * GDN_SCAN_CHUNK, which gdn_scan_backward reads; entries whose
 * token begins a request, or belongs to none, hold no meaning.
 */
typedef struct gdn_scan_args {
    int32_t batch;
    int32_t total_tokens;
    int32_t seq_len;        /* 0: packed; > 0: uniform */
    int32_t channels;
    int32_t num_state_rows; /* 0 means batch */
    int32_t act_dtype;      /* of x and o */
    int32_t gate_dtype;     /* of decay and beta: F32 or act_dtype */
    int32_t input_scale;    /* gdn_input_scale */
    uint32_t flags;         /* GDN_FLAG_BETA_SIGMOID or 0 */
    int64_t x_stride;
    int64_t decay_stride;
    int64_t beta_stride;
    int64_t o_stride;
    const void *x;
    const void *decay;
    const void *beta;        /* or NULL */
    void *o;
    const float *gate_bias;  /* [channels], with gate_scale, or NULL */
    const float *gate_scale; /* [channels] */
    const int32_t *cu_seqlens;
    const int32_t *seq_lens;
    const int32_t *slot_ids;
    const float *initial_state;
    float *final_state;
    float *chunk_states;
    int32_t *error_word;
} gdn_scan_args;

/* gdn_scan -- the recurrence, parallel over channels and along time: one launch,
 * no workspace, the same bits on every run.  For prefill and training.  total_tokens is at
 * most 2^31 - 8193 here and in gdn_scan_backward. */
gdn_status gdn_scan(const gdn_scan_args *args, gdn_stream stream);

/* gdn_scan_step -- the same result with the tokens of a request taken one after
 * another, for calls of one or a few tokens a request (chunk_states must be
 * NULL).  The arithmetic of a token is gdn_scan's. */
gdn_status gdn_scan_step(const gdn_scan_args *args, gdn_stream stream);

/*
 * gdn_scan_backward -- the gradient of gdn_scan, in one launch, with the same
 * bits on every run.  `forward` is the forward call: its o and final_state are
 * not used, its chunk_states are read (required when there are tokens).  Its
 * initial_state is read again and has to hold what the forward call found there: where
 * that call wrote its final states over it, pass a copy made before.  dh
 * being the gradient that reaches a token's state,
 *
 *     dh_t = d_o_t + a_{t+1} dh_{t+1}   (+ d_final_state[row] at a request's last token)
 *     dx   = n i dh,   d_beta = n x dh i'(beta)
 *     dg   = a h_{t-1} dh + n'(g) i x dh       (n'(g) taken as 0 where UNIT's n is 0)
 *     d_decay = dg,  or in the raw arm  dg gate_scale sigmoid(decay + gate_bias),
 *     d_gate_bias = sum over tokens of d_decay,  d_gate_scale = sum of dg softplus(decay + gate_bias)
 *     d_initial_state[row] = a dh at a request's first token (an empty request: d_final_state[row])
 *
 * The sums are kept in fp32 and written whole, over the tokens that requests own.
 * dx and d_o have act_dtype, d_decay and d_beta gate_dtype, the rest fp32.
 * d_final_state NULL is zero.  d_gate_bias, d_gate_scale and d_initial_state may
 * be NULL; dx, d_decay, and d_beta where there is a beta, are required.  Tokens
 * of no request and rows of none are not written.  Outputs overlap no input.
 */
typedef struct gdn_scan_grad_args {
    gdn_scan_args forward;
    int64_t d_o_stride; /* 0: channels, as in gdn_scan_args */
    int64_t dx_stride;
    int64_t d_decay_stride;
    int64_t d_beta_stride;
    const void *d_o;
    const float *d_final_state;
    void *dx;
    void *d_decay;
    void *d_beta;
    float *d_gate_bias;
    float *d_gate_scale;
    float *d_initial_state;
} gdn_scan_grad_args;

gdn_status gdn_scan_backward(const gdn_scan_grad_args *args, gdn_stream stream);

/*
 * gdn_rmsnorm -- residual addition and root-mean-square norm of each of `rows`
 * rows of `dim` values, all of it in fp32:
 *
 *     r = x + residual   (r = x without one),   residual_out = r in residual_dtype
 *     rstd = 1 / sqrt(mean(r^2) + eps),   y = r rstd weight
 *     out = y in x_dtype, or in E4M3 with scales:  s = max(|y|) / 448 over a row
 *     (group 0) or over each 128 columns (group 128; the last group of a row may be
 *     short), out = y / s, the maximum floored at 2^-100 so that s > 0.  y is formed as
 *     (r rstd) weight and the quotient rounded as a division's; the maximum of a whole row
 *     is max |r weight| times rstd (within three roundings of fp32 of max |y|).
 *
 * The norm takes r before residual_out is rounded.  x has x_stride elements from
 * row to row (0: dim); the other tensors are contiguous.  scales is fp32 [rows],
 * or [rows, ceil(dim / 128)]; rstd (NULL: not kept) is fp32 [rows], for
 * gdn_rmsnorm_backward.  residual_out may be residual.  dim is at most 2^20.
 */
typedef struct gdn_rmsnorm_args {
    int64_t rows;
    int32_t dim;
    int32_t x_dtype;
    int32_t residual_dtype; /* F32 or x_dtype */
    int32_t weight_dtype;   /* F32 or x_dtype */
    int32_t out_dtype;      /* x_dtype or E4M3 */
    int32_t group;          /* E4M3: 0 (a scale per row) or 128; else 0 */
    float eps;              /* >= 0 */
    int64_t x_stride;
    const void *x;
    const void *residual; /* or NULL */
    const void *weight;   /* [dim] */
    void *out;
    void *residual_out; /* with residual */
    float *scales;      /* with E4M3 */
    float *rstd;        /* or NULL */
} gdn_rmsnorm_args;

gdn_status gdn_rmsnorm(const gdn_rmsnorm_args *args, gdn_stream stream);

/*
 * gdn_rmsnorm_backward -- with r the norm's input as it was kept (residual_out, or
 * x), xhat = r rstd and d_residual the gradient that reaches residual_out from
 * elsewhere (NULL: none):
 *
 *     dx = rstd (weight d_out - xhat mean(weight d_out xhat)) + d_residual
 *     d_weight = sum over rows of d_out xhat
 *
 * dx is the gradient of x and of residual alike, for the rstd that is given: an fp32
 * rstd is up to 2^-22 off, which moves dx by up to 2^-22 (1 + 3 sqrt(dim)) rstd |weight d_out|
 * (on rows of one value that may be all of it).  r, d_residual and dx have
 * r_dtype, d_out x_dtype (d_out_stride elements from row to row; 0: dim), d_weight
 * is fp32.  dx may be d_residual.  Sums are fp32 and in a fixed order.  The
 * workspace is device memory of gdn_rmsnorm_backward_workspace_size() bytes,
 * 16-byte aligned (GDN_ERR_WORKSPACE otherwise); its contents are scratch.
 */
typedef struct gdn_rmsnorm_grad_args {
    int64_t rows;
    int32_t dim;
    int32_t x_dtype;
    int32_t r_dtype;      /* F32 or x_dtype */
    int32_t weight_dtype; /* F32 or x_dtype */
    int64_t d_out_stride;
    const void *d_out;
    const void *r;
    const void *weight;
    const float *rstd;
    const void *d_residual; /* or NULL */
    void *dx;
    float *d_weight; /* [dim] */
} gdn_rmsnorm_grad_args;

/* (size_t)-1 when the arguments are rejected (see gdn_last_error_message). */
size_t gdn_rmsnorm_backward_workspace_size(const gdn_rmsnorm_grad_args *args);
gdn_status gdn_rmsnorm_backward(const gdn_rmsnorm_grad_args *args, void *workspace, size_t workspace_bytes,
                                gdn_stream stream);

/*
 * gdn_grad_clip -- the norm of all elements of `count` tensors together, and the
 * tensors scaled to at most max_norm:
 *
 *     norm = sqrt(sum g^2),   out = g min(1, max_norm / (norm + eps))
 *
 * The arrays grads, outs, sizes and dtypes are HOST memory, read before the call
 * returns: device pointers, element counts (0: skipped) and gdn_dtypes (F32, F16,
 * BF16; an output has its gradient's).  outs[i] may be grads[i] (outs NULL: all in
 * place), and else overlaps neither it nor another; a tensor in place is written only if
 * it is scaled.  The squares and a
 * block's sum are fp32, joined in pairs of fp32, in a fixed order: the same bits on
 * every run (a norm above 1.8e19 counts as infinite).  norm is a device
 * float (or NULL).  A norm that is not finite scales nothing and sets
 * GDN_DEVERR_NONFINITE.  The workspace is device memory of
 * gdn_grad_clip_workspace_size() bytes, 16-byte aligned.
 */
typedef struct gdn_grad_clip_args {
    int32_t count;
    float max_norm; /* >= 0 */
    float eps;      /* >= 0 */
    const void *const *grads;
    void *const *outs;
    const int64_t *sizes;
    const int32_t *dtypes;
    float *norm;
    int32_t *error_word;
} gdn_grad_clip_args;

size_t gdn_grad_clip_workspace_size(const gdn_grad_clip_args *args);
gdn_status gdn_grad_clip(const gdn_grad_clip_args *args, void *workspace, size_t workspace_bytes, gdn_stream stream);

typedef enum gdn_activation {
    GDN_ACT_SILU = 0,      /* g sigmoid(g) */
    GDN_ACT_GELU = 1,      /* g Phi(g), by the error function */
    GDN_ACT_GELU_TANH = 2, /* g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2 */
    GDN_ACT_RELU = 3,      /* max(g, 0); its derivative at 0 is 0 */
    GDN_ACT_SIGMOID = 4    /* sigmoid(g) */
} gdn_activation;

/* Bytes of a row of gdn_glu's kept gates: the upper 16 bits of g and of u (inner rounded up
 * to a multiple of 64 of each), then the next 8 bits, 64 of g and the same 64 of u in turn. */
#define GDN_GLU_GATES_ROW(inner) (6 * (((int64_t)(inner) + 63) / 64 * 64))

/*
 * gdn_glu -- the gated half of a feed-forward block, both projections and what joins
 * them in one kernel, for each of `rows` tokens (with a launch before it that copies operands whose
 * rows are no words of 16 bytes, and one behind it where tiles are so few that K is cut):
 *
 *     g = x w_gate^T,   u = x w_up^T,   out = act(g) u
 *
 * x is [rows, dim] with x_stride elements from row to row (0: dim), out [rows, inner] with
 * out_stride (0: inner), the weights [inner, dim] contiguous, all of dtype F16 or BF16 (F32
 * is declined: GDN_ERR_UNSUPPORTED).  Products are summed in fp32 on the tensor cores, and
 * out is rounded once.  gates (NULL: not kept) receives g and u for gdn_glu_backward, cut to
 * 24 bits (sign, 8 bits of exponent, 15 of fraction; 16 would cost the gradients as much
 * again as their own roundings): GDN_GLU_GATES_ROW(inner) bytes a row, contiguous and
 * aligned to 16 bytes.  A few tokens (serving) take a kernel of their own.  out and gates
 * overlap no input and not one another (GDN_ERR_INVALID).
 *
 * The workspace is device memory of gdn_glu_workspace_size() bytes, 16-byte aligned (for
 * operands whose rows are no words of 16 bytes, and for shares of results where they are few);
 * its contents are scratch.  dim and inner are at most 2^20.
 */
typedef struct gdn_glu_args {
    int64_t rows;
    int32_t dim;
    int32_t inner;
    int32_t dtype;      /* F16 or BF16 */
    int32_t activation; /* gdn_activation */
    int64_t x_stride;
    int64_t out_stride;
    const void *x;
    const void *w_gate;
    const void *w_up;
    void *out;
    void *gates; /* or NULL */
    int32_t *error_word;
} gdn_glu_args;

/* (size_t)-1 when the arguments are rejected (see gdn_last_error_message). */
size_t gdn_glu_workspace_size(const gdn_glu_args *args);
gdn_status gdn_glu(const gdn_glu_args *args, void *workspace, size_t workspace_bytes, gdn_stream stream);

/*
 * gdn_glu_backward -- the gradient of gdn_glu for the gradient d_out of its output, at
 * the gates that it kept:
 *
 *     d_g = d_out u act'(g),   d_u = d_out act(g)
 *     dx = d_g w_gate + d_u w_up,   d_w_gate = d_g^T x,   d_w_up = d_u^T x
 *
 * d_g and d_u are formed in fp32 and rounded to dtype, as operands of the products (F16 with its
 * range: infinite above 65504, with fewer digits below 6e-5); sums
 * are fp32, in an order that the sizes and the device's number of SMs decide, whichever
 * gradients are wanted.  dx, and d_w_gate with d_w_up, may be NULL
 * (not wanted; what only they need may then be NULL too).  d_out_stride and dx_stride are
 * elements from row to row (0: without a gap); gates, the weights and their gradients are
 * contiguous.  Without rows the weights' gradients are zero.  Outputs overlap neither one
 * another nor what the products read, x, w_gate and w_up (GDN_ERR_INVALID); d_out and gates have been
 * read before an output is written.
 */
typedef struct gdn_glu_grad_args {
    int64_t rows;
    int32_t dim;
    int32_t inner;
    int32_t dtype;
    int32_t activation;
    int64_t x_stride;
    int64_t d_out_stride;
    int64_t dx_stride;
    const void *d_out;
    const void *x;
    const void *w_gate;
    const void *w_up;
    const void *gates;
    void *dx;       /* or NULL */
    void *d_w_gate; /* with d_w_up, or NULL */
    void *d_w_up;
    int32_t *error_word;
} gdn_glu_grad_args;

size_t gdn_glu_backward_workspace_size(const gdn_glu_grad_args *args);
gdn_status gdn_glu_backward(const gdn_glu_grad_args *args, void *workspace, size_t workspace_bytes, gdn_stream stream);

/* Elements that share a scale in 8-bit optimizer states. */
#define GDN_ADAMW_BLOCK 256

/*
 * gdn_adamw -- one AdamW step of `count` tensors.  With t the step's number (the first
 * is 1) and all of it in fp32:
 *
 *     k = min(1, max_norm / (*grad_norm + norm_eps))   (grad_norm given; else 1)
 *     m = beta1 m + (1 - beta1) k g,   v = beta2 v + (1 - beta2) (k g)^2
 *     p = p - lr (weight_decay p + (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps))
 *
 * grad_norm is a device float, the norm of all gradients: gdn_grad_clip with the largest
 * max_norm leaves them as they are and gives it, and the clip is then made here, where
 * they are read anyway.  A norm that is not finite leaves every tensor as it is and, where there
 * is one to step, sets GDN_DEVERR_NONFINITE.  (eps is rounded to fp32, but not to 0 unless it is.)
 *
 * The arrays are HOST memory, read before the call returns: device pointers, element
 * counts (0: skipped) and gdn_dtypes (F32, F16, BF16).  params, exp_avg (m), exp_avg_sq
 * (v) and their scales are updated in place; grads are read.  master (NULL: none, or
 * NULL for a tensor that has none) are fp32 copies of the weights: the step is then
 * taken on the copy, and params[i], which is not read, receives its rounding.  (A 16-bit
 * weight without a copy keeps nothing of a step that is less than half its last place.)  Tensors at
 * 16-byte addresses go by words; others, parts of a flat buffer say, element by element.
 *
 * state_dtype F32 keeps m and v as they are.  E4M3 keeps m and r = sqrt(v) in blocks of
 * GDN_ADAMW_BLOCK elements of a tensor (the last may be short), each with an fp32 scale
 * s = max(largest |m| (r), 2^-100) (1 / 448) in exp_avg_scales[i] (exp_avg_sq_scales[i]),
 * ceil(size / GDN_ADAMW_BLOCK) of them: the code is the quotient by s rounded to e4m3, and
 * of an r above zero at least the smallest, 2^-9, so that no step divides by the eps alone
 * where there was a gradient.  Each product, sum, root and quotient on the way there is
 * rounded to fp32 (k as max_norm times the reciprocal; a root of v below 2^-104, gradients of
 * 1e-15, may be off by a step of fp32).  The step itself takes m and v
 * before they are codes.  Codes and scales of zero are states of zero.  (A gradient that is
 * infinite or NaN makes both states of its block NaN, one whose square is beyond fp32 those of
 * exp_avg_sq, with a scale that is not finite; grad_norm keeps such a step from being taken.)
 *
 * step_device (or NULL) is the step's number in device memory, in place of `step`, and
 * lr_device the rate, in place of `lr`: a captured graph is replayed with new ones.  A
 * number below 1 there counts as 1.  (1 - beta^t is formed in fp32 of such a number, in 64 bits of
 * `step`: weights may differ in their last bits, states do not.)  No tensor overlaps another (GDN_ERR_INVALID where two
 * that are updated begin at one address: tied weights listed twice, say), but an F32 weight may be its own
 * copy in master.
 */
typedef struct gdn_adamw_args {
    int32_t count;
    int32_t state_dtype; /* F32 or E4M3 */
    int64_t step;        /* >= 1 */
    double lr;           /* >= 0 */
    double beta1, beta2; /* in [0, 1) */
    double eps;          /* >= 0 */
    double weight_decay; /* >= 0 */
    double max_norm;     /* >= 0, with grad_norm */
    double norm_eps;     /* >= 0, with grad_norm */
    void *const *params;
    const void *const *grads;
    void *const *exp_avg;
    void *const *exp_avg_sq;
    float *const *exp_avg_scales;    /* E4M3 */
    float *const *exp_avg_sq_scales; /* E4M3 */
    float *const *master;
    const int64_t *sizes;
    const int32_t *param_dtypes;
    const int32_t *grad_dtypes;
    const int64_t *step_device;
    const float *lr_device;
    const float *grad_norm;
    int32_t *error_word;
} gdn_adamw_args;

gdn_status gdn_adamw(const gdn_adamw_args *args, gdn_stream stream);

/* Static description of a status code ("ok", "invalid argument", ...). */
const char *gdn_status_string(gdn_status status);

/* Detail of the most recent non-OK status returned on this thread ("" if none). */
const char *gdn_last_error_message(void);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* GDN_H_ */
