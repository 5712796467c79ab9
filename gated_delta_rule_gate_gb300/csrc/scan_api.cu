// scan_api.cu -- the C entry points of the gated linear recurrence: host-side
// validation and dispatch.  Every check runs before anything is enqueued.
#include <cuda.h>  // CUtensorMap (the encoder is fetched through the runtime)

#include "launch.h"
#include "scan_cluster.cuh"
#include "scan_launch.h"
#include "status.h"

namespace {

using gdn::aligned;
using gdn::fail;
using gdn::scan::Args;

size_t size_of(int dt) { return dt == GDN_DTYPE_F32 ? 4 : 2; }

gdn_status check_types(const gdn_scan_args *a) {
    if (a->act_dtype != GDN_DTYPE_F32 && a->act_dtype != GDN_DTYPE_F16 && a->act_dtype != GDN_DTYPE_BF16)
        return fail(GDN_ERR_INVALID, "act_dtype: unknown dtype %d", a->act_dtype);
    if (a->gate_dtype != GDN_DTYPE_F32 && a->gate_dtype != a->act_dtype)
        return fail(GDN_ERR_INVALID, "gate_dtype must be F32 or the activation dtype");
    if (a->input_scale < GDN_INPUT_SCALE_NONE || a->input_scale > GDN_INPUT_SCALE_UNIT)
        return fail(GDN_ERR_INVALID, "unknown input_scale %d", a->input_scale);
    if (a->flags & ~GDN_FLAG_BETA_SIGMOID) return fail(GDN_ERR_INVALID, "unknown flag bits 0x%x", a->flags);
    if ((a->flags & GDN_FLAG_BETA_SIGMOID) && !a->beta)
        return fail(GDN_ERR_INVALID, "GDN_FLAG_BETA_SIGMOID given without beta");
    return GDN_OK;
}

gdn_status check_stride(int64_t stride, int channels, const char *what, int64_t *out) {
    if (stride != 0 && stride < channels)
        return fail(GDN_ERR_INVALID, "%s_stride (%lld) is less than channels (%d)", what, (long long)stride, channels);
    *out = stride ? stride : channels;
    return GDN_OK;
}

// q's rows begin on 16-byte addresses.
bool lines(const void *q, size_t e, int64_t stride) {
    return q == nullptr || (aligned(q, 16) && stride * (int64_t)e % 16 == 0);
}

// Sizes, token layout, gates, states and alignment, shared by every entry point.
// `needs_o`: the call writes o.
gdn_status validate(const gdn_scan_args *a, bool needs_o, Args *out) {
    if (!a) return fail(GDN_ERR_INVALID, "args is NULL");
    if (a->batch < 0) return fail(GDN_ERR_INVALID, "batch must be >= 0 (got %d)", a->batch);
    if (a->total_tokens < 0) return fail(GDN_ERR_INVALID, "total_tokens must be >= 0");
    if (a->channels <= 0) return fail(GDN_ERR_INVALID, "channels must be positive (got %d)", a->channels);
    if (a->channels > (1 << 24)) return fail(GDN_ERR_UNSUPPORTED, "more than 2^24 channels are not supported");
    gdn_status st = check_types(a);
    if (st != GDN_OK) return st;
    if (a->seq_len < 0) return fail(GDN_ERR_INVALID, "seq_len must be >= 0");
    if (a->seq_len > 0) {
        if (a->cu_seqlens) return fail(GDN_ERR_INVALID, "cu_seqlens requires the packed form; seq_len must be 0");
        if ((long long)a->batch * a->seq_len != a->total_tokens)
            return fail(GDN_ERR_INVALID, "uniform form: total_tokens (%d) != batch * seq_len (%d * %d)",
                        a->total_tokens, a->batch, a->seq_len);
    } else if (a->seq_lens) {
        return fail(GDN_ERR_INVALID, "seq_lens requires the uniform form; seq_len must be > 0");
    } else if (!a->cu_seqlens && a->batch > 0 && a->total_tokens % a->batch != 0) {
        return fail(GDN_ERR_INVALID, "uniform packing: total_tokens (%d) is not a multiple of batch (%d)",
                    a->total_tokens, a->batch);
    }
    if ((a->gate_bias == nullptr) != (a->gate_scale == nullptr))
        return fail(GDN_ERR_INVALID, "gate_bias and gate_scale must be given together (raw-gate arm) or not at all");
    if (a->num_state_rows < 0) return fail(GDN_ERR_INVALID, "num_state_rows must be >= 0");
    const int rows = a->num_state_rows ? a->num_state_rows : a->batch;
    if (!a->slot_ids && rows < a->batch)
        return fail(GDN_ERR_INVALID, "num_state_rows (%d) < batch (%d) without slot_ids", rows, a->batch);
    if (a->batch > 0 && a->total_tokens > 0 && (!a->x || !a->decay || (needs_o && !a->o)))
        return fail(GDN_ERR_INVALID, needs_o ? "x, decay and o are required" : "x and decay are required");
    Args &p = *out;
    if ((st = check_stride(a->x_stride, a->channels, "x", &p.xs)) != GDN_OK) return st;
    if ((st = check_stride(a->decay_stride, a->channels, "decay", &p.gs)) != GDN_OK) return st;
    if ((st = check_stride(a->beta_stride, a->channels, "beta", &p.bs)) != GDN_OK) return st;
    if ((st = check_stride(a->o_stride, a->channels, "o", &p.os)) != GDN_OK) return st;
    const size_t ea = size_of(a->act_dtype), eg = size_of(a->gate_dtype);
    if (!aligned(a->x, ea) || !aligned(a->o, ea) || !aligned(a->decay, eg) || !aligned(a->beta, eg) ||
        !aligned(a->gate_bias, 4) || !aligned(a->gate_scale, 4) || !aligned(a->cu_seqlens, 4) ||
        !aligned(a->seq_lens, 4) || !aligned(a->slot_ids, 4) || !aligned(a->initial_state, 4) ||
        !aligned(a->final_state, 4) || !aligned(a->chunk_states, 4) || !aligned(a->error_word, 4))
        return fail(GDN_ERR_INVALID, "a pointer is not aligned to its element size");
    p.B = a->batch;
    p.T = a->batch ? a->total_tokens : 0;  // without requests no kernel looks for a token's
    p.L = a->seq_len ? a->seq_len : (a->cu_seqlens || a->batch == 0 ? 0 : a->total_tokens / a->batch);
    p.D = a->channels;
    p.rows = rows;
    p.mode = a->input_scale;
    p.sigmoid = (a->flags & GDN_FLAG_BETA_SIGMOID) != 0;
    p.x = a->x, p.decay = a->decay, p.beta = a->beta, p.o = a->o;
    p.bias = a->gate_bias, p.scale = a->gate_scale;
    p.cu = a->cu_seqlens, p.seqlens = a->seq_lens, p.slots = a->slot_ids;
    p.init = a->initial_state, p.fin = a->final_state, p.chunk = a->chunk_states;
    p.err = a->error_word;
    p.wide = p.T > 0 && lines(a->x, ea, p.xs) && (!needs_o || lines(a->o, ea, p.os)) && lines(a->decay, eg, p.gs) &&
             lines(a->beta, eg, p.bs);
    return GDN_OK;
}

// The walks along time add up to three windows to a token's place.
gdn_status check_tokens(const Args &p) {
    constexpr int kMost = INT32_MAX - 4 * gdn::scan::kMaxWindow;
    if (p.T > kMost) return fail(GDN_ERR_UNSUPPORTED, "total_tokens above %d is not supported", kMost);
    return GDN_OK;
}

// Groups of four channels can be read and written as one word (gdn_scan_step).
bool four_wide(const Args &p, const gdn_scan_args *a) {
    const size_t ea = size_of(a->act_dtype), eg = size_of(a->gate_dtype);
    auto word = [](const void *q, size_t e, int64_t stride) {
        return q == nullptr || (aligned(q, 4 * e) && stride % 4 == 0);
    };
    return p.D % 4 == 0 && word(a->x, ea, p.xs) && word(a->o, ea, p.os) && word(a->decay, eg, p.gs) &&
           word(a->beta, eg, p.bs) && word(a->gate_bias, 4, 0) && word(a->gate_scale, 4, 0) &&
           word(a->initial_state, 4, 0) && word(a->final_state, 4, 0);
}

}  // namespace

extern "C" {

gdn_status gdn_scan(const gdn_scan_args *a, gdn_stream stream) {
    Args p;
    gdn_status st = validate(a, true, &p);
    if (st != GDN_OK || (st = check_tokens(p)) != GDN_OK) return st;
    if (p.B == 0) return gdn::ok();
    return gdn::cuda_status(gdn::scan::launch_scan(p, a->act_dtype, a->gate_dtype, (cudaStream_t)stream));
}

gdn_status gdn_scan_step(const gdn_scan_args *a, gdn_stream stream) {
    Args p;
    const gdn_status st = validate(a, true, &p);
    if (st != GDN_OK) return st;
    if (a->chunk_states) return fail(GDN_ERR_INVALID, "chunk_states are kept by gdn_scan only");
    if ((long long)p.B * p.D > (1LL << 37))
        return fail(GDN_ERR_UNSUPPORTED, "batch * channels exceeds 2^37");
    if (p.B == 0) return gdn::ok();
    return gdn::cuda_status(
        gdn::scan::launch_step(p, a->act_dtype, a->gate_dtype, four_wide(p, a), (cudaStream_t)stream));
}

gdn_status gdn_scan_backward(const gdn_scan_grad_args *a, gdn_stream stream) {
    if (!a) return fail(GDN_ERR_INVALID, "args is NULL");
    gdn::scan::GradArgs q;
    gdn_status st = validate(&a->forward, false, &q.f);
    if (st != GDN_OK || (st = check_tokens(q.f)) != GDN_OK) return st;
    Args &p = q.f;
    if ((st = check_stride(a->d_o_stride, p.D, "d_o", &q.dos)) != GDN_OK) return st;
    if ((st = check_stride(a->dx_stride, p.D, "dx", &q.dxs)) != GDN_OK) return st;
    if ((st = check_stride(a->d_decay_stride, p.D, "d_decay", &q.dgs)) != GDN_OK) return st;
    if ((st = check_stride(a->d_beta_stride, p.D, "d_beta", &q.dbs)) != GDN_OK) return st;
    if ((a->d_beta != nullptr) != (p.beta != nullptr))
        return fail(GDN_ERR_INVALID, p.beta ? "d_beta is required" : "d_beta given without beta");
    if ((a->d_gate_bias || a->d_gate_scale) && !p.bias)
        return fail(GDN_ERR_INVALID, "d_gate_bias and d_gate_scale belong to the raw-gate arm");
    if (p.B > 0 && p.T > 0) {
        if (!a->d_o || !a->dx || !a->d_decay) return fail(GDN_ERR_INVALID, "d_o, dx and d_decay are required");
        if (!p.chunk) return fail(GDN_ERR_INVALID, "chunk_states of the forward call are required");
    }
    const size_t ea = size_of(a->forward.act_dtype), eg = size_of(a->forward.gate_dtype);
    if (!aligned(a->d_o, ea) || !aligned(a->dx, ea) || !aligned(a->d_decay, eg) || !aligned(a->d_beta, eg) ||
        !aligned(a->d_final_state, 4) || !aligned(a->d_gate_bias, 4) || !aligned(a->d_gate_scale, 4) ||
        !aligned(a->d_initial_state, 4))
        return fail(GDN_ERR_INVALID, "a pointer is not aligned to its element size");
    q.d_o = a->d_o, q.dfin = a->d_final_state;
    q.dx = a->dx, q.dg = a->d_decay, q.db = a->d_beta;
    q.dbias = a->d_gate_bias, q.dscale = a->d_gate_scale, q.dinit = a->d_initial_state;
    p.fin = nullptr;
    p.o = nullptr;
    p.wide = p.wide && lines(a->d_o, ea, q.dos) && lines(a->dx, ea, q.dxs) && lines(a->d_decay, eg, q.dgs) &&
             lines(a->d_beta, eg, q.dbs);
    if (p.B == 0 && !q.dbias && !q.dscale) return gdn::ok();
    return gdn::cuda_status(
        gdn::scan::launch_grad(q, a->forward.act_dtype, a->forward.gate_dtype, (cudaStream_t)stream));
}

}  // extern "C"

namespace gdn {
namespace scan {

bool make_token_map(CUtensorMap *m, const void *base, int type, int64_t stride, int channels, int rows, int tokens) {
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                               const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
        return reinterpret_cast<Encode>(e == cudaSuccess && q == cudaDriverEntryPointSuccess ? ptr : nullptr);
    }();
    if (!encode) return false;
    const CUtensorMapDataType types[3] = {CU_TENSOR_MAP_DATA_TYPE_FLOAT32, CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                          CU_TENSOR_MAP_DATA_TYPE_BFLOAT16};
    const cuuint64_t dims[2] = {(cuuint64_t)channels, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * (type == 0 ? 4 : 2)};
    const cuuint32_t box[2] = {64, (cuuint32_t)tokens}, step[2] = {1, 1};
    return encode(m, types[type], 2, const_cast<void *>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_scan(const Args &p, int act, int gate, cudaStream_t stream) {
    const bool f = gate == GDN_DTYPE_F32;
    if (act == GDN_DTYPE_F32) return p.wide ? launch_scan_f32(p, stream) : launch_scan_f32_loose(p, stream);
    if (act == GDN_DTYPE_F16) return p.wide ? launch_scan_f16(p, f, stream) : launch_scan_f16_loose(p, f, stream);
    return p.wide ? launch_scan_bf16(p, f, stream) : launch_scan_bf16_loose(p, f, stream);
}

cudaError_t launch_grad(const GradArgs &p, int act, int gate, cudaStream_t stream) {
    const bool f = gate == GDN_DTYPE_F32, wide = p.f.wide;
    if (act == GDN_DTYPE_F32) return wide ? launch_grad_f32(p, stream) : launch_grad_f32_loose(p, stream);
    if (act == GDN_DTYPE_F16) return wide ? launch_grad_f16(p, f, stream) : launch_grad_f16_loose(p, f, stream);
    return wide ? launch_grad_bf16(p, f, stream) : launch_grad_bf16_loose(p, f, stream);
}

}  // namespace scan
}  // namespace gdn
