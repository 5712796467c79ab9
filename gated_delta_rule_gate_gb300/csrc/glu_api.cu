// glu_api.cu -- the C entry points of the gated feed-forward: host-side validation,
// the operands' tensor maps, and copies of operands whose rows are no words of 16 bytes.
#include <cuda.h>

#include <initializer_list>

#include "glu_launch.h"
#include "launch.h"
#include "overlap.h"
#include "ptx.cuh"
#include "status.h"

namespace gdn {
namespace glu {

// A map of rows for boxes of 128 bytes x `box` rows, 128-byte swizzle.
static bool make_map(CUtensorMap *m, const void *base, CUtensorMapDataType type, int rank, const cuuint64_t *dims,
                     const cuuint64_t *strides, int box) {
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
    const cuuint32_t wide = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 32 : type == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? 128 : 64;
    const cuuint32_t boxes[3] = {wide, (cuuint32_t)box, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode(m, type, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, boxes, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Of 16-bit rows.
static bool make_map(CUtensorMap *m, const void *base, bool bf16, int64_t stride, int64_t cols, int64_t rows, int box) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    return make_map(m, base, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, dims, strides,
                    box);
}
// Of fp32 shares [planes, rows, cols], for boxes of 32 rows.
static bool make_share_map(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int planes) {
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 4, (cuuint64_t)(cols * rows) * 4};
    return make_map(m, base, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, dims, strides, 32);
}

// Rows of `cols` 16-bit values, `from` elements apart, to rows `to` (a multiple of 8)
// elements apart at a 16-byte address; up to three operands a launch.
struct Copies {
    const uint16_t *src[3];
    uint16_t *dst[3];
    int64_t rows[3], from[3];
    int cols, to, count;
};
// 8 values a thread: read one by one (neighbours share their lines), written as a word.
__global__ void __launch_bounds__(256) spread_kernel(const __grid_constant__ Copies c) {
    ptx::grid_wait();
    const int per = c.to / 8;
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int64_t n = k < c.count ? c.rows[k] * per : 0;
        for (; i < n; i += (int64_t)gridDim.x * 256) {
            const int64_t row = i / per;
            const int at = (int)(i - row * per) * 8;
            const uint16_t *src = c.src[k] + row * c.from[k] + at;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = at + 2 * e < c.cols ? src[2 * e] : 0, hi = at + 2 * e + 1 < c.cols ? src[2 * e + 1] : 0;
                w[e] = lo | hi << 16;
            }
            *reinterpret_cast<uint4 *>(c.dst[k] + row * c.to + at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        i -= n;
    }
}

}  // namespace glu
}  // namespace gdn

namespace {

using namespace gdn::glu;
using gdn::aligned;
using gdn::fail;

constexpr int kMost = 1 << 20;
constexpr int kMostParts = 32;

int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }
int gate_columns(int inner) { return (inner + kGateColumns - 1) / kGateColumns * kGateColumns; }
static_assert(GDN_GLU_GATES_ROW(kGateColumns + 1) == gates_row(2 * kGateColumns), "the header's size of a row");
// Rows that a tensor map takes: words of 16 bytes.
bool lines(const void *p, int64_t stride) { return aligned(p, 16) && stride % 8 == 0; }
int64_t or_dense(int64_t stride, int64_t dense) { return stride ? stride : dense; }

gdn_status check_stride(int64_t stride, int least, const char *what) {
    if (stride != 0 && stride < least)
        return fail(GDN_ERR_INVALID, "%s (%lld) is less than a row (%d)", what, (long long)stride, least);
    return GDN_OK;
}
gdn_status check_sizes(int64_t rows, int dim, int inner, int dtype, int act) {
    if (rows < 0) return fail(GDN_ERR_INVALID, "rows must be >= 0");
    if (rows > (1LL << 31) - 512) return fail(GDN_ERR_UNSUPPORTED, "more than 2^31 - 512 rows are not supported");
    if (dim <= 0 || inner <= 0) return fail(GDN_ERR_INVALID, "dim and inner must be positive (got %d, %d)", dim, inner);
    if (dim > kMost || inner > kMost) return fail(GDN_ERR_UNSUPPORTED, "dim and inner above %d are not supported", kMost);
    if (dtype == GDN_DTYPE_F32) return fail(GDN_ERR_UNSUPPORTED, "dtype: the products take 16-bit operands, not float32");
    if (dtype != GDN_DTYPE_F16 && dtype != GDN_DTYPE_BF16) return fail(GDN_ERR_INVALID, "unknown dtype %d", dtype);
    // tiles of 256 x 128 results are counted in 32 bits, with up to 2 kMostParts of each
    if (((rows + 255) / 256) * ((inner + 127) / 128) >= 1LL << 25 || ((rows + 255) / 256) * ((dim + 127) / 128) >= 1LL << 25)
        return fail(GDN_ERR_UNSUPPORTED, "rows x inner or rows x dim is beyond 2^40");
    if (act < GDN_ACT_SILU || act > GDN_ACT_SIGMOID) return fail(GDN_ERR_INVALID, "unknown activation %d", act);
    return GDN_OK;
}

gdn_status validate(const gdn_glu_args *a) {
    if (!a) return fail(GDN_ERR_INVALID, "args is NULL");
    gdn_status st;
    if ((st = check_sizes(a->rows, a->dim, a->inner, a->dtype, a->activation)) != GDN_OK) return st;
    if ((st = check_stride(a->x_stride, a->dim, "x_stride")) != GDN_OK) return st;
    if ((st = check_stride(a->out_stride, a->inner, "out_stride")) != GDN_OK) return st;
    if (a->rows > 0 && (!a->x || !a->w_gate || !a->w_up || !a->out))
        return fail(GDN_ERR_INVALID, "x, w_gate, w_up and out are required");
    if (!aligned(a->x, 2) || !aligned(a->w_gate, 2) || !aligned(a->w_up, 2) || !aligned(a->out, 2) ||
        !aligned(a->error_word, 4))
        return fail(GDN_ERR_INVALID, "a pointer is not aligned to its element size");
    if (!aligned(a->gates, 16)) return fail(GDN_ERR_INVALID, "gates must be aligned to 16 bytes");
    return GDN_OK;
}
gdn_status validate_grad(const gdn_glu_grad_args *a) {
    if (!a) return fail(GDN_ERR_INVALID, "args is NULL");
    gdn_status st;
    if ((st = check_sizes(a->rows, a->dim, a->inner, a->dtype, a->activation)) != GDN_OK) return st;
    if ((st = check_stride(a->x_stride, a->dim, "x_stride")) != GDN_OK) return st;
    if ((st = check_stride(a->d_out_stride, a->inner, "d_out_stride")) != GDN_OK) return st;
    if ((st = check_stride(a->dx_stride, a->dim, "dx_stride")) != GDN_OK) return st;
    if ((a->d_w_gate == nullptr) != (a->d_w_up == nullptr))
        return fail(GDN_ERR_INVALID, "d_w_gate and d_w_up go together");
    if (a->d_w_gate && a->d_w_gate == a->d_w_up) return fail(GDN_ERR_INVALID, "d_w_gate and d_w_up are one tensor");
    if (!a->dx && !a->d_w_gate) return fail(GDN_ERR_INVALID, "dx, or d_w_gate and d_w_up, are required");
    if (a->rows > 0 && (!a->d_out || !a->gates)) return fail(GDN_ERR_INVALID, "d_out and gates are required");
    if (a->rows > 0 && a->dx && (!a->w_gate || !a->w_up)) return fail(GDN_ERR_INVALID, "w_gate and w_up are required");
    if (a->rows > 0 && a->d_w_gate && !a->x) return fail(GDN_ERR_INVALID, "x is required");
    if (!aligned(a->x, 2) || !aligned(a->w_gate, 2) || !aligned(a->w_up, 2) || !aligned(a->d_out, 2) ||
        !aligned(a->dx, 2) || !aligned(a->d_w_gate, 2) || !aligned(a->d_w_up, 2) ||
        !aligned(a->error_word, 4))
        return fail(GDN_ERR_INVALID, "a pointer is not aligned to its element size");
    if (!aligned(a->gates, 16)) return fail(GDN_ERR_INVALID, "gates must be aligned to 16 bytes");
    return GDN_OK;
}

// A workspace given out piece by piece, in multiples of 256 bytes (before it is known to suffice).
struct Pieces {
    unsigned char *base;
    size_t used = 0;
    void *take(int64_t values) {
        void *p = reinterpret_cast<void *>(reinterpret_cast<uintptr_t>(base) + used);
        used += ((size_t)values * 2 + 255) / 256 * 256;
        return p;
    }
};
// An operand as a tensor map takes it: itself, or a copy.
struct Operand {
    const void *at;
    int64_t stride, cols, rows;
    const void *from = nullptr;  // what is copied, and its rows' distance
    int64_t from_stride = 0;
};
Operand operand(const void *p, int64_t rows, int64_t cols, int64_t stride, Pieces *ws) {
    Operand o = {p, stride, cols, rows};
    if (lines(p, stride)) return o;
    o.from = p, o.from_stride = stride, o.stride = padded(cols);
    o.at = ws->take(rows * o.stride);
    return o;
}
// Those of up to three operands of one width that are copies are made.
cudaError_t bring(std::initializer_list<const Operand *> operands, cudaStream_t s) {
    Copies c = {};
    int64_t n = 0;
    for (const Operand *o : operands) {
        if (!o->from) continue;
        const int k = c.count++;
        c.src[k] = static_cast<const uint16_t *>(o->from);
        c.dst[k] = static_cast<uint16_t *>(const_cast<void *>(o->at));
        c.rows[k] = o->rows, c.from[k] = o->from_stride;
        c.cols = (int)o->cols, c.to = (int)o->stride;
        n += o->rows * (o->stride / 8);
    }
    if (c.count == 0) return cudaSuccess;
    const int64_t blocks = (n + 255) / 256, most = (int64_t)gdn::sm_count() * 16;
    return gdn::launch_early(spread_kernel, (unsigned)(blocks < most ? blocks : most), 256, 0, s, c);
}
bool map_of(CUtensorMap *m, const Operand &o, bool bf16, int box) {
    return make_map(m, o.at, bf16, o.stride, o.cols, o.rows, box);
}
// A result of job.rows rows, by tensor map where its rows are words of 16 bytes and end with
// one: a store that is cut inside a word writes all of it.  (A load is cut where it should be.)
bool result(Result *r, const Job &job, void *at, int64_t stride, int cols, bool bf16) {
    r->at = at, r->stride = stride, r->by_map = lines(at, stride) && cols % 8 == 0;
    return !r->by_map || make_map(&r->map, at, bf16, stride, cols, job.rows, 32);
}
// `results` results of rows x cols in tiles of 256 x width, sums over `pairs` pairs of operands with
// `depth` of K each, in `parts` stretches.
void sizes(Job *j, int64_t rows, int cols, int width, int results, int64_t depth, int pairs, int parts) {
    j->rows = rows, j->cols = cols, j->results = results, j->pairs = pairs, j->parts = parts;
    j->tiles_m = (int)((rows + 255) / 256), j->tiles_n = (cols + width - 1) / width;
    j->blocks_k = (int)((depth + 63) / 64);
    j->per_part = (pairs * j->blocks_k + parts - 1) / parts;
    j->tiles = (uint32_t)j->tiles_m * (uint32_t)j->tiles_n * (uint32_t)(results * parts);
}
// The stretches that K of results is cut into: those that make the device's
// time least, in K-steps (0.27 us) of a pair of blocks.  A tile costs some six steps beside its
// own; shares are written and read in fp32, and a launch is added.  Pairs of blocks take
// tiles in turn, the first job's first, so the longest time is that of the first pair, or of
// the first one that has a tile less of the first job.  (64 tokens x 4096 x 1024 fp16, 8 tiles: 14.1 us in
// eight stretches, 24.5 in one; 256 x 4096 x 8192, 64 tiles, stays in one, 31.)
struct Cut {
    int64_t tiles = 0, steps = 0;  // in one stretch
    double values = 0;             // of all results
    // into n stretches that are worth it: of eight steps at least, none of them empty, and
    // not where the tiles alone fill the device four times
    bool into(int n, int64_t device) const {
        if (n == 1) return true;
        const int64_t per = (steps + n - 1) / n;
        return tiles > 0 && tiles < 4 * device && steps / n >= 8 && (steps + per - 1) / per == n;
    }
};
void choose_parts(const Cut &first, const Cut &second, int *n1, int *n2) {
    static const int counts[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, kMostParts};
    const int64_t device = gdn::sm_count() / 2;
    double least = -1;
    for (const int i : counts) {
        if (!first.into(i, device)) continue;
        for (const int j : counts) {
            if (!second.into(j, device)) continue;
            const int64_t a = first.tiles * i, all = a + second.tiles * j;
            const double ta = (double)((first.steps + i - 1) / i + 6), tb = (double)((second.steps + j - 1) / j + 6);
            double longest = 0;
            for (const int64_t p : {(int64_t)0, a % device}) {
                const int64_t mine = (a - p + device - 1) / device, total = (all - p + device - 1) / device;
                const double t = (double)mine * ta + (double)(total - mine) * tb;
                if (t > longest) longest = t;
            }
            const double shares = (i > 1 ? first.values * i : 0) + (j > 1 ? second.values * j : 0);
            if (shares > 0) longest += 12 + shares * 8 / 6.5e6 / 0.27;
            if (least < 0 || longest < least) least = longest, *n1 = i, *n2 = j;
        }
    }
}
Cut cut_of(int64_t rows, int cols, int results, int64_t depth, int pairs) {
    Cut c;
    c.tiles = (rows + 255) / 256 * ((cols + 255) / 256) * results;
    c.steps = (depth + 63) / 64 * pairs;
    c.values = (double)rows * padded(cols) * results;
    return c;
}
Join join_of(const Job &j, const void *shares) {
    Join r = {};
    r.shares = static_cast<const float *>(shares);
    r.rows = j.rows, r.stride = j.c[0].stride, r.cols = j.cols, r.cs = (int)padded(j.cols);
    r.parts = j.parts, r.results = j.results;
    r.words = j.cols % 4 == 0 && r.stride % 4 == 0;
    for (int z = 0; z < j.results; ++z) r.out[z] = j.c[z].at, r.words = r.words && aligned(j.c[z].at, 8);
    return r;
}
gdn_status no_map() { return fail(GDN_ERR_CUDA, "a tensor map could not be made"); }

struct ForwardPlan {
    bool few;
    Operand x, wg, wu;
    int parts;
    void *shares;
    size_t bytes;
};
ForwardPlan plan(const gdn_glu_args *a, void *ws) {
    ForwardPlan f = {};
    f.few = a->rows <= kFewTokens;
    if (f.few || a->rows == 0) return f;
    Pieces pieces = {static_cast<unsigned char *>(ws)};
    f.x = operand(a->x, a->rows, a->dim, or_dense(a->x_stride, a->dim), &pieces);
    f.wg = operand(a->w_gate, a->inner, a->dim, a->dim, &pieces);
    f.wu = operand(a->w_up, a->inner, a->dim, a->dim, &pieces);
    Cut cut;
    cut.tiles = (a->rows + 255) / 256 * ((a->inner + 127) / 128);
    cut.steps = (a->dim + 63) / 64;
    cut.values = 2.0 * (double)a->rows * padded(a->inner);
    int none;
    choose_parts(cut, Cut(), &f.parts, &none);
    f.shares = pieces.take(f.parts > 1 ? 4 * a->rows * padded(a->inner) * f.parts : 0);
    f.bytes = pieces.used;
    return f;
}

struct BackwardPlan {
    Operand x, wg, wu, dg, du;
    int in_parts, w_parts;
    void *in_shares, *w_shares;
    size_t bytes;
};
BackwardPlan plan_grad(const gdn_glu_grad_args *a, void *ws) {
    BackwardPlan b = {};
    if (a->rows == 0) return b;
    Pieces pieces = {static_cast<unsigned char *>(ws)};
    const int64_t F = a->inner, Fp = padded(F), Dp = padded(a->dim);
    b.dg = {pieces.take(a->rows * Fp), Fp, F, a->rows};
    b.du = {pieces.take(a->rows * Fp), Fp, F, a->rows};
    if (a->d_w_gate) b.x = operand(a->x, a->rows, a->dim, or_dense(a->x_stride, a->dim), &pieces);
    if (a->dx) {
        b.wg = operand(a->w_gate, F, a->dim, a->dim, &pieces);
        b.wu = operand(a->w_up, F, a->dim, a->dim, &pieces);
    }
    // As if all gradients were wanted, whichever are: the order of a gradient's sum is promised not
    // to depend on that.
    choose_parts(cut_of(a->rows, a->dim, 1, F, 2), cut_of(F, a->dim, 2, a->rows, 1), &b.in_parts, &b.w_parts);
    b.in_shares = pieces.take(a->dx && b.in_parts > 1 ? 2 * a->rows * Dp * b.in_parts : 0);
    b.w_shares = pieces.take(a->d_w_gate && b.w_parts > 1 ? 4 * F * Dp * b.w_parts : 0);
    b.bytes = pieces.used;
    return b;
}

// Results that the kernels write while they still read what they would lie on.
struct Operands {
    const char *name;
    gdn::Span span;
};
gdn_status check_apart(std::initializer_list<Operands> results, std::initializer_list<Operands> read) {
    for (const Operands *r = results.begin(); r != results.end(); ++r) {
        for (const Operands &o : read)
            if (gdn::overlap(r->span, o.span)) return fail(GDN_ERR_INVALID, "%s overlaps %s", r->name, o.name);
        for (const Operands *o = r + 1; o != results.end(); ++o)
            if (gdn::overlap(r->span, o->span)) return fail(GDN_ERR_INVALID, "%s overlaps %s", r->name, o->name);
    }
    return GDN_OK;
}
// (A distance that no memory has room for stays within 64 bits.)
gdn::Span span_of(const void *p, int64_t rows, int64_t stride, int cols) {
    const int64_t s = or_dense(stride, cols), most = (1LL << 61) / (rows > 0 ? rows : 1);
    return {p, rows, 2 * (s < most ? s : most), 2 * (int64_t)cols};
}

gdn_status check_workspace(const void *ws, size_t have, size_t need) {
    if (need > 0 && (ws == nullptr || have < need || !aligned(ws, 16)))
        return fail(GDN_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned (got %zu)", need, have);
    return GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_glu_workspace_size(const gdn_glu_args *a) {
    if (validate(a) != GDN_OK) return (size_t)-1;
    gdn::ok();
    return plan(a, nullptr).bytes;
}

gdn_status gdn_glu(const gdn_glu_args *a, void *ws, size_t ws_bytes, gdn_stream stream) {
    gdn_status st = validate(a);
    if (st != GDN_OK) return st;
    const ForwardPlan f = plan(a, ws);
    if ((st = check_workspace(ws, ws_bytes, f.bytes)) != GDN_OK) return st;
    if (a->rows == 0) return gdn::ok();
    const int64_t weight = 2 * (int64_t)a->inner * a->dim;
    st = check_apart({{"out", span_of(a->out, a->rows, a->out_stride, a->inner)},
                      {"gates", gdn::block_of(a->gates, a->rows * gates_row(gate_columns(a->inner)))}},
                     {{"x", span_of(a->x, a->rows, a->x_stride, a->dim)},
                      {"w_gate", gdn::block_of(a->w_gate, weight)},
                      {"w_up", gdn::block_of(a->w_up, weight)}});
    if (st != GDN_OK) return st;
    const bool bf16 = a->dtype == GDN_DTYPE_BF16;
    const int64_t os = or_dense(a->out_stride, a->inner);
    cudaStream_t s = (cudaStream_t)stream;
    if (f.few) {
        Few p = {};
        p.x = a->x, p.wg = a->w_gate, p.wu = a->w_up, p.out = a->out, p.gates = static_cast<unsigned char *>(a->gates);
        p.xs = or_dense(a->x_stride, a->dim), p.os = os;
        p.T = (int)a->rows, p.D = a->dim, p.F = a->inner, p.Fg = gate_columns(a->inner), p.act = a->activation;
        p.words = lines(a->x, p.xs) && lines(a->w_gate, a->dim) && lines(a->w_up, a->dim);
        return gdn::cuda_status(bf16 ? launch_few_bf16(p, s) : launch_few_f16(p, s));
    }
    ForwardArgs p = {};
    Job &j = p.job;
    sizes(&j, a->rows, a->inner, 128, 1, a->dim, 1, f.parts);
    p.act = a->activation, p.err = a->error_word;
    const int Fg = gate_columns(a->inner);
    if (!map_of(&j.a[0], f.x, bf16, 128) || !map_of(&j.b[0], f.wg, bf16, 128) || !map_of(&j.b[1], f.wu, bf16, 128) ||
        !result(&j.c[0], j, a->out, os, a->inner, bf16))
        return no_map();
    if (a->gates) {
        unsigned char *gates = static_cast<unsigned char *>(a->gates);
        for (int i = 0; i < 2; ++i)
            if (!result(&j.c[1 + i], j, gates + i * 2 * (int64_t)Fg, gates_row(Fg) / 2, Fg, bf16)) return no_map();
        const cuuint64_t dims[2] = {2 * (cuuint64_t)Fg, (cuuint64_t)a->rows}, strides[1] = {(cuuint64_t)gates_row(Fg)};
        if (!make_map(&p.lower, gates + 4 * (int64_t)Fg, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, dims, strides, 32))
            return no_map();
    }
    if (j.parts > 1 && !make_share_map(&j.shares, f.shares, padded(a->inner), a->rows, 2 * j.parts)) return no_map();
    cudaError_t e = bring({&f.x, &f.wg, &f.wu}, s);
    if (e == cudaSuccess) e = bf16 ? launch_forward_bf16(p, a->gates, s) : launch_forward_f16(p, a->gates, s);
    if (e == cudaSuccess && j.parts > 1) {
        ForwardJoin q = {};
        q.shares = static_cast<const float *>(f.shares), q.out = a->out, q.gates = static_cast<unsigned char *>(a->gates);
        q.rows = a->rows, q.os = os, q.F = a->inner, q.cs = (int)padded(a->inner), q.Fg = Fg;
        q.parts = j.parts, q.act = a->activation;
        q.words = a->inner % 4 == 0 && os % 4 == 0 && aligned(a->out, 8);
        e = bf16 ? launch_forward_join_bf16(q, s) : launch_forward_join_f16(q, s);
    }
    return gdn::cuda_status(e);
}

size_t gdn_glu_backward_workspace_size(const gdn_glu_grad_args *a) {
    if (validate_grad(a) != GDN_OK) return (size_t)-1;
    gdn::ok();
    return plan_grad(a, nullptr).bytes;
}

gdn_status gdn_glu_backward(const gdn_glu_grad_args *a, void *ws, size_t ws_bytes, gdn_stream stream) {
    gdn_status st = validate_grad(a);
    if (st != GDN_OK) return st;
    const BackwardPlan b = plan_grad(a, ws);
    if ((st = check_workspace(ws, ws_bytes, b.bytes)) != GDN_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t T = a->rows;
    const int D = a->dim, F = a->inner;
    // d_out and gates have been read before any result is written
    const int64_t weight = 2 * (int64_t)F * D;
    st = check_apart({{"dx", span_of(a->dx, T, a->dx_stride, D)},
                      {"d_w_gate", gdn::block_of(a->d_w_gate, weight)},
                      {"d_w_up", gdn::block_of(a->d_w_up, weight)}},
                     {{"x", span_of(a->d_w_gate ? a->x : nullptr, T, a->x_stride, D)},
                      {"w_gate", gdn::block_of(a->dx && T ? a->w_gate : nullptr, weight)},
                      {"w_up", gdn::block_of(a->dx && T ? a->w_up : nullptr, weight)}});
    if (st != GDN_OK) return st;
    cudaError_t e = cudaSuccess;
    if (T == 0) {  // sums over nothing
        const size_t bytes = (size_t)F * D * 2;
        if (a->d_w_gate) e = cudaMemsetAsync(a->d_w_gate, 0, bytes, s);
        if (a->d_w_up && e == cudaSuccess) e = cudaMemsetAsync(a->d_w_up, 0, bytes, s);
        return gdn::cuda_status(e);
    }
    const bool bf16 = a->dtype == GDN_DTYPE_BF16;
    Backward p = {};
    Job &in = p.job[0], &w = p.job[1];
    Joins joins = {};
    p.err = a->error_word;
    if (a->dx) {
        sizes(&in, T, D, 256, 1, F, 2, b.in_parts);
        if (!map_of(&in.a[0], b.dg, bf16, 128) || !map_of(&in.a[1], b.du, bf16, 128) ||
            !map_of(&in.b[0], b.wg, bf16, 64) || !map_of(&in.b[1], b.wu, bf16, 64) ||
            !result(&in.c[0], in, a->dx, or_dense(a->dx_stride, D), D, bf16) ||
            (in.parts > 1 && !make_share_map(&in.shares, b.in_shares, padded(D), T, in.parts)))
            return no_map();
        if (in.parts > 1) joins.j[joins.count++] = join_of(in, b.in_shares);
    }
    if (a->d_w_gate) {
        sizes(&w, F, D, 256, 2, T, 1, b.w_parts);
        w.a_outer = 1;
        if (!map_of(&w.a[0], b.dg, bf16, 64) || !map_of(&w.a[1], b.du, bf16, 64) || !map_of(&w.b[0], b.x, bf16, 64) ||
            !result(&w.c[0], w, a->d_w_gate, D, D, bf16) || !result(&w.c[1], w, a->d_w_up, D, D, bf16) ||
            (w.parts > 1 && !make_share_map(&w.shares, b.w_shares, padded(D), F, 2 * w.parts)))
            return no_map();
        if (w.parts > 1) joins.j[joins.count++] = join_of(w, b.w_shares);
    }
    GateGrad g = {};
    g.d_out = a->d_out, g.gates = static_cast<const unsigned char *>(a->gates);
    g.dg = const_cast<void *>(b.dg.at), g.du = const_cast<void *>(b.du.at);
    g.rows = T, g.dos = or_dense(a->d_out_stride, F), g.F = F, g.Fp = (int)padded(F), g.Fg = gate_columns(F);
    g.act = a->activation;
    g.words = F % 8 == 0 && lines(a->d_out, g.dos);
    e = bf16 ? launch_gate_grad_bf16(g, s) : launch_gate_grad_f16(g, s);
    if (e == cudaSuccess) e = bring({&b.x, &b.wg, &b.wu}, s);
    if (e == cudaSuccess) e = bf16 ? launch_backward_bf16(p, s) : launch_backward_f16(p, s);
    if (e == cudaSuccess && joins.count) e = bf16 ? launch_join_bf16(joins, s) : launch_join_f16(joins, s);
    return gdn::cuda_status(e);
}

}  // extern "C"
