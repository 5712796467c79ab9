// layer_binding.cpp -- Python entry points of the recurrent-layer operators, over
// torch tensors.
//
// As the ctypes binding of the other entry points, these functions read shapes,
// strides, dtypes and pointers, fill the C structs of include/gdn.h and call the
// library on the current stream (or `stream`); what they allocate when an output is
// not given is torch memory of that stream.  They are C++ because a decode step is
// over in the time that Python takes to look at ten tensors (8.7 us a call from
// Python).  The library's functions are handed in by bind(): this module links to
// Python and torch alone, both loaded already.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <optional>
#include <string>
#include <vector>

#include "../../include/gdn.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

constexpr int64_t kChunk = GDN_SCAN_CHUNK;

struct Library {
    decltype(&gdn_scan) scan;
    decltype(&gdn_scan_step) step;
    decltype(&gdn_scan_backward) backward;
    decltype(&gdn_rmsnorm) norm;
    decltype(&gdn_rmsnorm_backward) norm_backward;
    decltype(&gdn_rmsnorm_backward_workspace_size) norm_workspace;
    decltype(&gdn_grad_clip) clip;
    decltype(&gdn_grad_clip_workspace_size) clip_workspace;
} lib;
PyObject *check_status, *scan_gradients, *norm_result, *norm_gradients, *stream_handle_name;

[[noreturn]] void refuse(PyObject *type, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(type, fmt, ap);
    va_end(ap);
    throw python_error();
}

void done(gdn_status status) {
    if (status == GDN_OK) return;
    PyObject *r = PyObject_CallFunction(check_status, "i", (int)status);  // raises with the library's message
    Py_XDECREF(r);
    throw python_error();
}

// ---------------------------------------------------------------- arguments
// A function's parameters: the first `positional` by place or by name, the rest by
// name; the first `required` have no default (None).
struct Signature {
    const char *function;
    int positional, required;
    std::vector<const char *> names;
    std::vector<PyObject *> interned;
};
constexpr int kMost = 24;

void parse(Signature &s, PyObject *const *args, Py_ssize_t n, PyObject *kwnames, PyObject **out) {
    const int count = (int)s.names.size();
    if (n > s.positional)
        refuse(PyExc_TypeError, "%s() takes %d positional arguments but %zd were given", s.function, s.positional, n);
    for (int i = 0; i < count; ++i) out[i] = i < n ? args[i] : nullptr;
    const Py_ssize_t named = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t k = 0; k < named; ++k) {
        PyObject *name = PyTuple_GET_ITEM(kwnames, k);
        int at = -1;
        for (int i = 0; i < count && at < 0; ++i)
            if (s.interned[i] == name) at = i;
        for (int i = 0; i < count && at < 0; ++i)
            if (PyUnicode_Compare(s.interned[i], name) == 0) at = i;
        if (at < 0) refuse(PyExc_TypeError, "%s() got an unexpected keyword argument '%U'", s.function, name);
        if (out[at]) refuse(PyExc_TypeError, "%s() got multiple values for argument '%U'", s.function, name);
        out[at] = args[n + k];
    }
    for (int i = 0; i < s.required; ++i)
        if (!out[i]) refuse(PyExc_TypeError, "%s() missing required argument '%s'", s.function, s.names[i]);
    for (int i = 0; i < count; ++i)
        if (out[i] == Py_None) out[i] = nullptr;
}

const Tensor *tensor(PyObject *o, const char *what) {
    if (!o) return nullptr;
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", what);
    return &THPVariable_Unpack(o);
}
const Tensor &needed(PyObject *o, const char *what) {
    const Tensor *t = tensor(o, what);
    if (!t) refuse(PyExc_TypeError, "%s must be a tensor", what);
    return *t;
}
bool flag(PyObject *o) {
    if (!o) return false;
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}
int32_t whole(PyObject *o, const char *what) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred() && !PyErr_ExceptionMatches(PyExc_OverflowError)) throw python_error();
    PyErr_Clear();
    if (v < 1 || v > INT32_MAX) refuse(PyExc_ValueError, "%s must be in [1, 2^31)", what);
    return (int32_t)v;
}
double number(PyObject *o, double otherwise) {
    if (!o) return otherwise;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

int code(const Tensor &t, const char *what) {
    switch (t.scalar_type()) {
        case ScalarType::Float: return GDN_DTYPE_F32;
        case ScalarType::Half: return GDN_DTYPE_F16;
        case ScalarType::BFloat16: return GDN_DTYPE_BF16;
        default: refuse(PyExc_TypeError, "%s: unsupported dtype %s", what, c10::toString(t.scalar_type()));
    }
}
std::string text(IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + ")";
}
void check_device(const Tensor &t, const char *what) {
    if (!t.is_cuda())
        refuse(PyExc_ValueError, "libgdn takes device tensors; %s is on %s", what, t.device().str().c_str());
}
// All tensors of a call lie where `first` does (which is refused with a message of its
// own where that is no device).
struct Named {
    const Tensor *t;
    const char *what;
};
void one_device(const Tensor &first, std::initializer_list<Named> others) {
    if (!first.is_cuda()) return;
    const c10::Device device = first.device();
    for (const Named &o : others)
        if (o.t && o.t->device() != device && o.t->is_cuda())
            refuse(PyExc_ValueError, "%s is on %s, not on %s as the rest of the call's device tensors", o.what,
                   o.t->device().str().c_str(), device.str().c_str());
}
void check(const Tensor &t, ScalarType type, const char *what) {
    check_device(t, what);
    if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s", what, c10::toString(type));
}
void check_shape(const Tensor &t, IntArrayRef shape, const char *what) {
    if (t.sizes() != shape)
        refuse(PyExc_ValueError, "%s must be %s, got %s", what, text(shape).c_str(), text(t.sizes()).c_str());
}
// Address of a contiguous device tensor of the given type, or null.
template <typename T = void>
T *address(const Tensor *t, ScalarType type, const char *what) {
    if (!t) return nullptr;
    check(*t, type, what);
    if (!t->is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", what);
    return static_cast<T *>(t->data_ptr());
}
template <typename T = void>
T *address(const Tensor *t, ScalarType type, const char *what, IntArrayRef shape) {
    if (t) check_shape(*t, shape, what);
    return address<T>(t, type, what);
}
struct Rows {
    void *at;
    int64_t stride;
};
// Address and elements between rows of a device tensor whose last dimension is
// contiguous and whose leading ones lie in it as one; rows do not overlap.
Rows rows(const Tensor *t, ScalarType type, IntArrayRef shape, const char *what) {
    if (!t) return {nullptr, 0};
    check(*t, type, what);
    check_shape(*t, shape, what);
    const int64_t dim = t->dim(), last = dim ? shape[dim - 1] : 1;
    if (t->is_contiguous()) return {t->data_ptr(), last};
    if (t->stride(-1) != 1 && last != 1) refuse(PyExc_ValueError, "%s must have contiguous channels", what);
    int64_t step = last, count = 1;  // of the dimensions so far; those of one have no stride
    for (int64_t d = dim - 2; d >= 0; --d) {
        if (shape[d] == 1) continue;
        if (count == 1) step = t->stride(d);
        else if (t->stride(d) != count * step) refuse(PyExc_ValueError, "%s must have one stride over all its rows", what);
        count *= shape[d];
    }
    // a step of 0 is the library's word for rows without a gap
    if (step < last) refuse(PyExc_ValueError, "%s has rows that overlap (an expanded tensor?): pass a copy", what);
    return {t->data_ptr(), step};
}
Rows rows(const Tensor &t, ScalarType type, IntArrayRef shape, const char *what) { return rows(&t, type, shape, what); }

// The stream of a call: the current one of the tensors' device, a torch stream, or a
// handle.  While it lives, that device is the current one and memory is made for that stream.
class Stream {
  public:
    Stream(PyObject *o, const Tensor &like) : Stream(o, like.device()) {}
    Stream(PyObject *o, c10::Device home) {
        if (!home.is_cuda()) return;  // refused with a message of its own
        const c10::DeviceIndex device = home.index();
        if (!o) {
            handle_ = c10::cuda::getCurrentCUDAStream(device).stream();
            // the library launches on the current device
            if (device != c10::cuda::current_device()) device_.emplace(device);
            return;
        }
        PyObject *held = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttr(o, stream_handle_name);
        if (!held) throw python_error();
        void *h = PyLong_AsVoidPtr(held);
        Py_DECREF(held);
        if (!h && PyErr_Occurred()) throw python_error();
        handle_ = static_cast<cudaStream_t>(h);
        guard_.emplace(c10::cuda::getStreamFromExternal(handle_, device));
    }
    gdn_stream get() const { return reinterpret_cast<gdn_stream>(handle_); }

  private:
    cudaStream_t handle_ = nullptr;
    std::optional<c10::cuda::CUDAStreamGuard> guard_;
    std::optional<c10::cuda::CUDAGuard> device_;
};

at::TensorOptions on(const Tensor &like, ScalarType type) { return at::TensorOptions().device(like.device()).dtype(type); }
// Device memory by torch's allocator (past the dispatcher, 0.3 us a tensor).
Tensor make(IntArrayRef shape, c10::Device device, ScalarType type) {
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
}
Tensor make(IntArrayRef shape, const Tensor &like, ScalarType type) { return make(shape, like.device(), type); }

// The call wrote into these given tensors: autograd is to notice where it has kept one.
void written(std::initializer_list<const Tensor *> ts) {
    for (const Tensor *t : ts)
        if (t && t->defined() && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

PyObject *wrap(const Tensor &t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }
// A named tuple of the tensors (None where undefined).
PyObject *tuple_of(PyObject *cls, std::initializer_list<const Tensor *> ts) {
    PyObject *args[8];
    size_t n = 0;
    for (const Tensor *t : ts) args[n++] = t ? wrap(*t) : Py_NewRef(Py_None);
    PyObject *r = PyObject_Vectorcall(cls, args, n, nullptr);
    while (n) Py_XDECREF(args[--n]);
    return r;
}

// ---------------------------------------------------------------- scan
// Parameters that gdn_scan, gdn_scan_step and gdn_scan_backward share, by place.
struct ScanCall {
    const Tensor *x, *decay, *beta, *bias, *scale, *cu, *seq_lens, *slots, *init, *fin;
    PyObject *input_scale;
    bool sigmoid;
    const Tensor *err;
};

gdn_scan_args scan_args(const ScanCall &c, const Tensor *out, const Tensor *chunks) {
    constexpr ScalarType f32 = ScalarType::Float, i32 = ScalarType::Int;
    const Tensor &x = *c.x, &decay = *c.decay;
    one_device(x, {{&decay, "decay"}, {c.beta, "beta"}, {c.bias, "gate_bias"}, {c.scale, "gate_scale"},
                   {c.cu, "cu_seqlens"}, {c.seq_lens, "seq_lens"}, {c.slots, "slot_ids"}, {c.init, "initial_state"},
                   {c.fin, "final_state"}, {c.err, "error_word"}, {out, "out"}, {chunks, "chunk_states"}});
    gdn_scan_args a = {};
    a.act_dtype = code(x, "x");
    a.gate_dtype = code(decay, "decay");
    const IntArrayRef shape = x.sizes();
    int64_t B, T;
    if (shape.size() == 2) {
        T = shape[0];
        B = c.cu ? c.cu->numel() - 1 : 1;
        if (B < 0) refuse(PyExc_ValueError, "cu_seqlens must have batch + 1 entries");
    } else if (shape.size() == 3) {
        B = shape[0];
        a.seq_len = (int32_t)shape[1];
        T = B * shape[1];
        if (c.cu) refuse(PyExc_ValueError, "cu_seqlens goes with packed tokens, x [tokens, channels]");
    } else {
        refuse(PyExc_ValueError, "x must be [tokens, channels] or [batch, tokens, channels]");
    }
    const int64_t D = shape.back();
    if (T > INT32_MAX || B > INT32_MAX || D > INT32_MAX)
        refuse(PyExc_ValueError, "x has more than 2^31 - 1 tokens or channels");
    a.batch = (int32_t)B, a.total_tokens = (int32_t)T, a.channels = (int32_t)D;
    if (c.input_scale) {
        const char *s = PyUnicode_Check(c.input_scale) ? PyUnicode_AsUTF8(c.input_scale) : "";
        if (s && !strcmp(s, "lerp")) a.input_scale = GDN_INPUT_SCALE_LERP;
        else if (s && !strcmp(s, "unit")) a.input_scale = GDN_INPUT_SCALE_UNIT;
        else if (!s || strcmp(s, "none"))
            refuse(PyExc_ValueError, "input_scale must be one of none, lerp, unit");
    }
    a.flags = c.sigmoid ? GDN_FLAG_BETA_SIGMOID : 0;
    const ScalarType act = x.scalar_type(), gate = decay.scalar_type();
    const Rows xr = rows(x, act, shape, "x"), gr = rows(decay, gate, shape, "decay");
    const Rows br = rows(c.beta, gate, shape, "beta"), orow = rows(out, act, shape, "out");
    a.x = xr.at, a.x_stride = xr.stride;
    a.decay = gr.at, a.decay_stride = gr.stride;
    a.beta = br.at, a.beta_stride = br.stride;
    a.o = orow.at, a.o_stride = orow.stride;
    const Tensor *state = c.init ? c.init : c.fin;
    if (state) {
        if (state->dim() != 2 || state->size(1) != D)
            refuse(PyExc_ValueError, "states must be [rows, %lld]", (long long)D);
        if (state->size(0) == 0 && B > 0) refuse(PyExc_ValueError, "states of %lld requests have no rows", (long long)B);
        if (state->size(0) > INT32_MAX) refuse(PyExc_ValueError, "more than 2^31 - 1 state rows");
        a.num_state_rows = (int32_t)state->size(0);
        a.initial_state = address<const float>(c.init, f32, "initial_state");
        a.final_state = address<float>(c.fin, f32, "final_state", state->sizes());
    } else if (c.slots) {
        a.num_state_rows = INT32_MAX;  // no states, no rows for an id to be beyond
    }
    const int64_t d[1] = {D}, b[1] = {B}, ch[2] = {(T + kChunk - 1) / kChunk, D};
    a.gate_bias = address<const float>(c.bias, f32, "gate_bias", d);
    a.gate_scale = address<const float>(c.scale, f32, "gate_scale", d);
    a.cu_seqlens = address<const int32_t>(c.cu, i32, "cu_seqlens");
    a.seq_lens = address<const int32_t>(c.seq_lens, i32, "seq_lens", b);
    // rows of no tokens the library knows as packed ones; all requests are empty
    if (shape.size() == 3 && !a.seq_len) a.seq_lens = nullptr;
    a.slot_ids = address<const int32_t>(c.slots, i32, "slot_ids", b);
    a.chunk_states = address<float>(chunks, f32, "chunk_states", ch);
    a.error_word = address<int32_t>(c.err, i32, "error_word");
    return a;
}

Signature scan_signature = {"gdn_scan", 2, 2, {"x", "decay", "beta", "gate_bias", "gate_scale", "beta_sigmoid",
                            "input_scale", "cu_seqlens", "seq_lens", "slot_ids", "initial_state", "final_state", "out",
                            "want_chunk_states", "error_word", "stream"}, {}};
Signature step_signature = {"gdn_scan_step", 2, 2, {"x", "decay", "beta", "gate_bias", "gate_scale", "beta_sigmoid",
                            "input_scale", "cu_seqlens", "seq_lens", "slot_ids", "initial_state", "final_state", "out",
                            "error_word", "stream"}, {}};

ScanCall scan_call(PyObject **v, PyObject *err) {
    ScanCall c;
    c.x = &needed(v[0], "x"), c.decay = &needed(v[1], "decay"), c.beta = tensor(v[2], "beta");
    c.bias = tensor(v[3], "gate_bias"), c.scale = tensor(v[4], "gate_scale"), c.sigmoid = flag(v[5]);
    c.input_scale = v[6], c.cu = tensor(v[7], "cu_seqlens"), c.seq_lens = tensor(v[8], "seq_lens");
    c.slots = tensor(v[9], "slot_ids"), c.init = tensor(v[10], "initial_state");
    c.fin = tensor(v[11], "final_state"), c.err = tensor(err, "error_word");
    return c;
}

PyObject *py_scan(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kwnames) {
    HANDLE_TH_ERRORS
    PyObject *v[kMost];
    parse(scan_signature, args, n, kwnames, v);
    const ScanCall c = scan_call(v, v[14]);
    const bool keep = flag(v[13]);
    const Tensor &x = *c.x, *given = tensor(v[12], "out");
    gdn_scan_args a = scan_args(c, given, nullptr);
    Stream stream(v[15], x);
    Tensor out, chunks;
    if (!given) {
        out = make(x.sizes(), x, x.scalar_type());
        a.o = out.data_ptr(), a.o_stride = 0;
    }
    if (keep) {
        chunks = make({(a.total_tokens + kChunk - 1) / kChunk, a.channels}, x, ScalarType::Float);
        a.chunk_states = chunks.data_ptr<float>();
    }
    done(lib.scan(&a, stream.get()));
    written({given, c.fin});
    PyObject *o = given ? Py_NewRef(v[12]) : THPVariable_Wrap(out);
    return keep ? Py_BuildValue("(NN)", o, THPVariable_Wrap(chunks)) : o;
    END_HANDLE_TH_ERRORS
}

PyObject *py_step(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kwnames) {
    HANDLE_TH_ERRORS
    PyObject *v[kMost];
    parse(step_signature, args, n, kwnames, v);
    const ScanCall c = scan_call(v, v[13]);
    const Tensor &x = *c.x, *given = tensor(v[12], "out");
    gdn_scan_args a = scan_args(c, given, nullptr);
    Stream stream(v[14], x);
    Tensor out;
    if (!given) {
        out = make(x.sizes(), x, x.scalar_type());
        a.o = out.data_ptr(), a.o_stride = 0;
    }
    done(lib.step(&a, stream.get()));
    written({given, c.fin});
    return given ? Py_NewRef(v[12]) : THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

Signature backward_signature = {"gdn_scan_backward", 4, 4, {"d_out", "x", "decay", "chunk_states", "beta", "gate_bias",
                                "gate_scale", "beta_sigmoid", "input_scale", "cu_seqlens", "seq_lens", "slot_ids",
                                "initial_state", "d_final_state", "dx", "d_decay", "d_beta", "d_gate_bias",
                                "d_gate_scale", "d_initial_state", "error_word", "stream", "num_state_rows"}, {}};

PyObject *py_backward(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kwnames) {
    HANDLE_TH_ERRORS
    constexpr ScalarType f32 = ScalarType::Float;
    PyObject *v[kMost];
    parse(backward_signature, args, n, kwnames, v);
    const Tensor &dout = needed(v[0], "d_out"), *chunks = &needed(v[3], "chunk_states");
    ScanCall c;
    c.x = &needed(v[1], "x"), c.decay = &needed(v[2], "decay"), c.beta = tensor(v[4], "beta");
    c.bias = tensor(v[5], "gate_bias"), c.scale = tensor(v[6], "gate_scale"), c.sigmoid = flag(v[7]);
    c.input_scale = v[8], c.cu = tensor(v[9], "cu_seqlens"), c.seq_lens = tensor(v[10], "seq_lens");
    c.slots = tensor(v[11], "slot_ids"), c.init = tensor(v[12], "initial_state");
    c.err = tensor(v[20], "error_word");
    const Tensor *dfin = tensor(v[13], "d_final_state");
    c.fin = c.init ? nullptr : dfin;  // gives the number of state rows
    const Tensor &x = *c.x, &decay = *c.decay;
    gdn_scan_grad_args a = {};
    a.forward = scan_args(c, nullptr, chunks);
    a.forward.final_state = nullptr;
    const Tensor *state = c.init ? c.init : dfin ? dfin : tensor(v[19], "d_initial_state");
    if (state && state->dim() == 2 && state->size(0) == 0 && a.forward.batch > 0)
        refuse(PyExc_ValueError, "states of %d requests have no rows", a.forward.batch);
    if (v[22]) {
        const int32_t n = whole(v[22], "num_state_rows");
        if (state && state->dim() == 2 && state->size(0) != n)
            refuse(PyExc_ValueError, "num_state_rows is %d, the states have %lld", n, (long long)state->size(0));
        a.forward.num_state_rows = n;
    }
    const IntArrayRef shape = x.sizes();
    const ScalarType act = x.scalar_type(), gate = decay.scalar_type();
    auto given = [&](int i, const char *what) {
        const Tensor *t = tensor(v[i], what);
        return t ? *t : Tensor();
    };
    auto some = [](const Tensor &t) { return t.defined() ? &t : nullptr; };
    Tensor dx = given(14, "dx"), dg = given(15, "d_decay"), db = given(16, "d_beta");
    Tensor dbias = given(17, "d_gate_bias"), dscale = given(18, "d_gate_scale"), dinit = given(19, "d_initial_state");
    one_device(x, {{&dout, "d_out"}, {dfin, "d_final_state"}, {some(dx), "dx"}, {some(dg), "d_decay"},
                   {some(db), "d_beta"}, {some(dbias), "d_gate_bias"}, {some(dscale), "d_gate_scale"},
                   {some(dinit), "d_initial_state"}});
    const Rows dor = rows(dout, act, shape, "d_out");
    Rows dxr = rows(some(dx), act, shape, "dx"), dgr = rows(some(dg), gate, shape, "d_decay");
    Rows dbr = rows(some(db), gate, shape, "d_beta");
    Stream stream(v[21], x);
    // every token and row is written unless requests may leave some out
    const bool whole = !c.cu && !c.seq_lens && !c.slots;
    auto token = [&](Tensor &t, Rows &r, ScalarType type) {
        if (t.defined()) return;
        t = whole ? make(shape, x, type) : at::zeros(shape, on(x, type));
        r.at = t.data_ptr();
    };
    token(dx, dxr, act);
    token(dg, dgr, gate);
    if (c.beta) token(db, dbr, gate);
    if (c.bias && !dbias.defined()) dbias = make(c.bias->sizes(), x, f32);
    if (c.bias && !dscale.defined()) dscale = make(c.bias->sizes(), x, f32);
    if (c.init && !dinit.defined()) dinit = at::zeros(c.init->sizes(), on(x, f32));
    a.d_o = dor.at, a.d_o_stride = dor.stride;
    a.dx = dxr.at, a.dx_stride = dxr.stride;
    a.d_decay = dgr.at, a.d_decay_stride = dgr.stride;
    a.d_beta = dbr.at, a.d_beta_stride = dbr.stride;
    const int64_t d[1] = {shape.back()};
    a.d_gate_bias = address<float>(some(dbias), f32, "d_gate_bias", d);
    a.d_gate_scale = address<float>(some(dscale), f32, "d_gate_scale", d);
    if (c.init || dfin) {
        a.d_final_state = address<const float>(dfin, f32, "d_final_state", state->sizes());
        a.d_initial_state = address<float>(some(dinit), f32, "d_initial_state", state->sizes());
    } else if (dinit.defined()) {
        if (dinit.dim() != 2 || dinit.size(1) != d[0])
            refuse(PyExc_ValueError, "d_initial_state must be [rows, %lld]", (long long)d[0]);
        a.forward.num_state_rows = (int32_t)dinit.size(0);
        a.d_initial_state = address<float>(&dinit, f32, "d_initial_state");
    }
    done(lib.backward(&a, stream.get()));
    for (int i = 14; i < 20; ++i) written({tensor(v[i], "a gradient")});
    return tuple_of(scan_gradients, {&dx, &dg, &db, &dbias, &dscale, &dinit});
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- norm
Signature norm_signature = {"gdn_rmsnorm", 2, 2, {"x", "weight", "residual", "eps", "out_dtype", "group", "want_rstd",
                            "out", "residual_out", "scales", "stream"}, {}};

PyObject *py_norm(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kwnames) {
    HANDLE_TH_ERRORS
    constexpr ScalarType f32 = ScalarType::Float;
    PyObject *v[kMost];
    parse(norm_signature, args, n, kwnames, v);
    const Tensor &x = needed(v[0], "x"), &weight = needed(v[1], "weight"), *residual = tensor(v[2], "residual");
    const ScalarType type = x.scalar_type();
    ScalarType out_type = type;
    if (v[4]) {
        if (!THPDtype_Check(v[4])) refuse(PyExc_TypeError, "out_dtype must be a torch dtype");
        out_type = reinterpret_cast<THPDtype *>(v[4])->scalar_type;
    }
    const bool e4m3 = out_type == ScalarType::Float8_e4m3fn;
    gdn_rmsnorm_args a = {};
    a.x_dtype = code(x, "x");
    a.residual_dtype = residual ? code(*residual, "residual") : a.x_dtype;
    a.weight_dtype = code(weight, "weight");
    a.out_dtype = e4m3 ? GDN_DTYPE_E4M3 : (out_type == type ? a.x_dtype : -1);
    a.group = (int32_t)number(v[5], 0);
    a.eps = (float)number(v[3], 1e-6);
    const IntArrayRef shape = x.sizes();
    const int64_t D = shape.empty() ? 0 : shape.back();
    if (D > INT32_MAX) refuse(PyExc_ValueError, "x has more than 2^31 - 1 columns");
    a.dim = (int32_t)D;
    a.rows = D ? x.numel() / D : 0;
    const Tensor *o = tensor(v[7], "out"), *ro = tensor(v[8], "residual_out"), *sc = tensor(v[9], "scales");
    if (ro && !residual) refuse(PyExc_ValueError, "residual_out given without residual");
    one_device(x, {{&weight, "weight"}, {residual, "residual"}, {o, "out"}, {ro, "residual_out"}, {sc, "scales"}});
    const Rows xr = rows(x, type, shape, "x");
    a.x = xr.at, a.x_stride = xr.stride;
    const int64_t d[1] = {D};
    a.weight = address(&weight, weight.scalar_type(), "weight", d);
    std::vector<int64_t> scales_shape(shape.begin(), shape.empty() ? shape.end() : shape.end() - 1);
    const std::vector<int64_t> lead = scales_shape;
    if (a.group) scales_shape.push_back((D + 127) / 128);
    Stream stream(v[10], x);
    Tensor out, res_out, scales, rstd;
    out = o ? *o : make(shape, x, out_type);
    if (residual) {
        const ScalarType rt = residual->scalar_type();
        a.residual = address(residual, rt, "residual", shape);
        res_out = ro ? *ro : make(shape, x, rt);
        a.residual_out = address(&res_out, rt, "residual_out", shape);
    }
    if (e4m3 || sc) {
        scales = sc ? *sc : make(scales_shape, x, f32);
        a.scales = address<float>(&scales, f32, "scales", scales_shape);
    }
    if (flag(v[6])) {
        rstd = make(lead, x, f32);
        a.rstd = rstd.data_ptr<float>();
    }
    a.out = address(&out, out_type, "out", shape);
    done(lib.norm(&a, stream.get()));
    written({o, ro, sc});
    return tuple_of(norm_result, {&out, &res_out, &scales, &rstd});
    END_HANDLE_TH_ERRORS
}

// A workspace may have any type and shape.
const Tensor *workspace(PyObject *o) {
    const Tensor *t = tensor(o, "workspace");
    if (!t) return nullptr;
    check_device(*t, "workspace");
    if (!t->is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
    return t;
}
// Device memory of `need` bytes where `given` is none.
struct Workspace {
    Tensor t;
    void *at;
    size_t bytes;
    Workspace(const Tensor *given, size_t need, const Tensor &like) {
        if (need == (size_t)-1) need = 0;  // the call says what is wrong
        t = given ? *given : make({(int64_t)need}, like, ScalarType::Byte);
        at = t.data_ptr();
        bytes = t.numel() * t.element_size();
    }
};

Signature norm_backward_signature = {"gdn_rmsnorm_backward", 4, 4, {"d_out", "r", "weight", "rstd", "d_residual", "dx",
                                     "d_weight", "workspace", "stream"}, {}};

PyObject *py_norm_backward(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kwnames) {
    HANDLE_TH_ERRORS
    constexpr ScalarType f32 = ScalarType::Float;
    PyObject *v[kMost];
    parse(norm_backward_signature, args, n, kwnames, v);
    const Tensor &dout = needed(v[0], "d_out"), &r = needed(v[1], "r"), &weight = needed(v[2], "weight");
    const Tensor &rstd = needed(v[3], "rstd"), *dres = tensor(v[4], "d_residual"), *dxg = tensor(v[5], "dx");
    const Tensor *dwg = tensor(v[6], "d_weight");
    const Tensor *given = workspace(v[7]);
    one_device(r, {{&dout, "d_out"}, {&weight, "weight"}, {&rstd, "rstd"}, {dres, "d_residual"}, {dxg, "dx"},
                   {dwg, "d_weight"}, {given, "workspace"}});
    gdn_rmsnorm_grad_args a = {};
    const IntArrayRef shape = r.sizes();
    const ScalarType rt = r.scalar_type();
    const int64_t D = shape.empty() ? 0 : shape.back();
    if (D > INT32_MAX) refuse(PyExc_ValueError, "r has more than 2^31 - 1 columns");
    a.dim = (int32_t)D;
    a.rows = D ? r.numel() / D : 0;
    a.x_dtype = code(dout, "d_out"), a.r_dtype = code(r, "r"), a.weight_dtype = code(weight, "weight");
    const Rows dr = rows(dout, dout.scalar_type(), shape, "d_out");
    const int64_t d[1] = {D};
    a.d_out = dr.at, a.d_out_stride = dr.stride;
    a.r = address(&r, rt, "r");
    a.weight = address(&weight, weight.scalar_type(), "weight", d);
    a.rstd = address<const float>(&rstd, f32, "rstd", shape.empty() ? shape : shape.slice(0, shape.size() - 1));
    a.d_residual = address(dres, rt, "d_residual", shape);
    Stream stream(v[8], r);
    Tensor dx = dxg ? *dxg : make(shape, r, rt), dw = dwg ? *dwg : make(d, r, f32);
    a.dx = address(&dx, rt, "dx", shape);
    a.d_weight = address<float>(&dw, f32, "d_weight", d);
    const Workspace ws(given, given ? 0 : lib.norm_workspace(&a), r);
    done(lib.norm_backward(&a, ws.at, ws.bytes, stream.get()));
    written({dxg, dwg});
    return tuple_of(norm_gradients, {&dx, &dw});
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- clip
Signature clip_signature = {"gdn_grad_clip", 2, 2, {"grads", "max_norm", "eps", "out", "norm", "error_word",
                            "workspace", "stream"}, {}};

// The items of a sequence, held while it lives.
struct Sequence {
    PyObject *s;
    Py_ssize_t n;
    Sequence(PyObject *o, const char *what) : s(PySequence_Fast(o, what)) {
        if (!s) throw python_error();
        n = PySequence_Fast_GET_SIZE(s);
    }
    Sequence(const Sequence &) = delete;
    ~Sequence() { Py_DECREF(s); }
    const Tensor &at(Py_ssize_t i, const char *what) const { return needed(PySequence_Fast_GET_ITEM(s, i), what); }
};

PyObject *py_clip(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kwnames) {
    HANDLE_TH_ERRORS
    PyObject *v[kMost];
    parse(clip_signature, args, n, kwnames, v);
    if (!v[0]) refuse(PyExc_TypeError, "grads must be a sequence of tensors");
    if (!v[1]) refuse(PyExc_TypeError, "max_norm must be a number");
    const double max_norm = number(v[1], 0), eps = number(v[2], 1e-6);
    const Sequence grads(v[0], "grads must be a sequence of tensors");
    std::optional<Sequence> outs;
    if (v[3]) {
        outs.emplace(v[3], "out must be a sequence of tensors");
        if (outs->n != grads.n)
            refuse(PyExc_ValueError, "out must have a tensor for each of the %zd gradients", grads.n);
    }
    std::vector<const void *> in(grads.n);
    std::vector<void *> to(grads.n);
    std::vector<int64_t> sizes(grads.n);
    std::vector<int32_t> types(grads.n);
    const Tensor *given_norm = tensor(v[4], "norm"), *given = workspace(v[6]), *err = tensor(v[5], "error_word");
    if (grads.n)
        one_device(grads.at(0, "a gradient"), {{given_norm, "norm"}, {err, "error_word"}, {given, "workspace"}});
    else if (given_norm)
        one_device(*given_norm, {{err, "error_word"}, {given, "workspace"}});
    for (Py_ssize_t i = 0; i < grads.n; ++i) {
        const Tensor &g = grads.at(i, "a gradient");
        one_device(grads.at(0, "a gradient"), {{&g, "a gradient"}, {outs ? &outs->at(i, "an output") : nullptr, "an output"}});
        types[i] = code(g, "a gradient");
        in[i] = address(&g, g.scalar_type(), "a gradient");
        sizes[i] = g.numel();
        if (outs) to[i] = address(&outs->at(i, "an output"), g.scalar_type(), "an output", g.sizes());
    }
    const c10::Device device = grads.n      ? grads.at(0, "a gradient").device()
                               : given_norm ? given_norm->device()
                                            : c10::Device(at::kCUDA, c10::cuda::current_device());
    Stream stream(v[7], device);
    Tensor norm = given_norm ? *given_norm : make({1}, device, ScalarType::Float);
    gdn_grad_clip_args a = {};
    a.count = (int32_t)grads.n;
    a.max_norm = (float)max_norm;
    a.eps = (float)eps;
    a.grads = in.data(), a.outs = outs ? to.data() : nullptr, a.sizes = sizes.data(), a.dtypes = types.data();
    const int64_t one[1] = {1};
    a.norm = address<float>(&norm, ScalarType::Float, "norm", one);
    a.error_word = address<int32_t>(err, ScalarType::Int, "error_word");
    const Workspace ws(given, given ? 0 : lib.clip_workspace(&a), norm);
    done(lib.clip(&a, ws.at, ws.bytes, stream.get()));
    for (Py_ssize_t i = 0; i < grads.n; ++i) written({outs ? &outs->at(i, "an output") : &grads.at(i, "a gradient")});
    written({given_norm});
    return THPVariable_Wrap(norm);
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- module
// bind(addresses of the library's functions, check, ScanGradients, NormResult, NormGradients)
PyObject *py_bind(PyObject *, PyObject *args) {
    HANDLE_TH_ERRORS
    unsigned long long f[8];
    PyObject *objects[4];
    if (!PyArg_ParseTuple(args, "(KKKKKKKK)OOOO", f, f + 1, f + 2, f + 3, f + 4, f + 5, f + 6, f + 7, objects,
                          objects + 1, objects + 2, objects + 3))
        return nullptr;
    lib.scan = reinterpret_cast<decltype(lib.scan)>(f[0]);
    lib.step = reinterpret_cast<decltype(lib.step)>(f[1]);
    lib.backward = reinterpret_cast<decltype(lib.backward)>(f[2]);
    lib.norm = reinterpret_cast<decltype(lib.norm)>(f[3]);
    lib.norm_backward = reinterpret_cast<decltype(lib.norm_backward)>(f[4]);
    lib.norm_workspace = reinterpret_cast<decltype(lib.norm_workspace)>(f[5]);
    lib.clip = reinterpret_cast<decltype(lib.clip)>(f[6]);
    lib.clip_workspace = reinterpret_cast<decltype(lib.clip_workspace)>(f[7]);
    check_status = Py_NewRef(objects[0]), scan_gradients = Py_NewRef(objects[1]);
    norm_result = Py_NewRef(objects[2]), norm_gradients = Py_NewRef(objects[3]);
    stream_handle_name = PyUnicode_InternFromString("cuda_stream");
    for (Signature *s : {&scan_signature, &step_signature, &backward_signature, &norm_signature,
                         &norm_backward_signature, &clip_signature}) {
        if (!s->interned.empty()) continue;
        for (const char *name : s->names) s->interned.push_back(PyUnicode_InternFromString(name));
    }
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS

PyMethodDef methods[] = {
    {"gdn_scan", FAST(py_scan),
     "gdn_scan($module, x, decay, *, beta=None, gate_bias=None, gate_scale=None, beta_sigmoid=False, "
     "input_scale='none', cu_seqlens=None, seq_lens=None, slot_ids=None, initial_state=None, final_state=None, "
     "out=None, want_chunk_states=False, error_word=None, stream=None)\n--\n\n"
     "The gated linear recurrence over whole sequences, per channel\n\n"
     "    g = decay, or gate_scale * softplus(decay + gate_bias);  a = exp(g)\n"
     "    h_t = a h_{t-1} + n i x_t;  out_t = h_t\n\n"
     "with i = 1, beta or sigmoid(beta) and n = 1, 1 - a (\"lerp\") or sqrt(1 - a^2)\n"
     "(\"unit\").  x, decay and beta are [T, D] packed (requests by cu_seqlens, else one)\n"
     "or [B, S, D] (seq_lens bounds the rows); they may be columns of wider tensors.\n"
     "States are fp32 [rows, D], row slot_ids[b] or b; final_state is written if given\n"
     "and may be initial_state; without states slot_ids only tell which requests to skip\n"
     "(negative ones).  Returns out (allocated when not given; tokens of no\n"
     "request are not written), or (out, chunk_states) with want_chunk_states, for\n"
     "gdn_scan_backward."},
    {"gdn_scan_step", FAST(py_step),
     "gdn_scan_step($module, x, decay, *, beta=None, gate_bias=None, gate_scale=None, beta_sigmoid=False, "
     "input_scale='none', cu_seqlens=None, seq_lens=None, slot_ids=None, initial_state=None, final_state=None, "
     "out=None, error_word=None, stream=None)\n--\n\n"
     "gdn_scan for one or a few tokens a request (time grows with the longest): the\n"
     "serving step, usually with initial_state and final_state one slab that slot_ids\n"
     "address."},
    {"gdn_scan_backward", FAST(py_backward),
     "gdn_scan_backward($module, d_out, x, decay, chunk_states, *, beta=None, gate_bias=None, gate_scale=None, "
     "beta_sigmoid=False, input_scale='none', cu_seqlens=None, seq_lens=None, slot_ids=None, initial_state=None, "
     "d_final_state=None, dx=None, d_decay=None, d_beta=None, d_gate_bias=None, d_gate_scale=None, "
     "d_initial_state=None, error_word=None, stream=None, num_state_rows=None)\n--\n\n"
     "Gradients of gdn_scan for the gradient d_out of its output (and d_final_state of\n"
     "its final states): the forward call's arguments and the chunk_states that it\n"
     "returned (initial_state as that call found it: keep a copy of one that it wrote its\n"
     "final states over).  Returns ScanGradients(dx, d_decay, d_beta, d_gate_bias, d_gate_scale,\n"
     "d_initial_state), None where there is no such input.  Outputs are allocated when\n"
     "not given (zeros where tokens or state rows may belong to no request); a given\n"
     "one is not written there.  num_state_rows says how many rows the forward call's\n"
     "states had where none are given here: without it only a negative slot id is a bad\n"
     "one, as in a forward call without states."},
    {"gdn_rmsnorm", FAST(py_norm),
     "gdn_rmsnorm($module, x, weight, *, residual=None, eps=1e-06, out_dtype=None, group=0, want_rstd=False, "
     "out=None, residual_out=None, scales=None, stream=None)\n--\n\n"
     "r = x + residual; out = r / sqrt(mean(r^2) + eps) * weight over the last dimension,\n"
     "in fp32.  out_dtype is x's, or torch.float8_e4m3fn with fp32 scales (out * scale is\n"
     "the value): one per row (group 0) or per 128 columns (128).  Returns\n"
     "NormResult(out, residual, scales, rstd): residual is r in residual's dtype (float32\n"
     "or x's; residual_out may be residual), rstd is for gdn_rmsnorm_backward; None where\n"
     "there is none or it was not asked for."},
    {"gdn_rmsnorm_backward", FAST(py_norm_backward),
     "gdn_rmsnorm_backward($module, d_out, r, weight, rstd, *, d_residual=None, dx=None, d_weight=None, "
     "workspace=None, stream=None)\n--\n\n"
     "Gradients of gdn_rmsnorm for the gradient d_out of its (unquantised) output and\n"
     "d_residual of the residual that it returned; r is that residual (x where there was\n"
     "none), rstd what it returned.  Returns NormGradients(dx, dweight): dx, in r's dtype,\n"
     "is the gradient of x and of residual alike (dx may be d_residual); dweight is\n"
     "float32."},
    {"gdn_grad_clip", FAST(py_clip),
     "gdn_grad_clip($module, grads, max_norm, *, eps=1e-06, out=None, norm=None, error_word=None, workspace=None, "
     "stream=None)\n--\n\n"
     "The 2-norm of all elements of the tensors grads together, and each scaled by\n"
     "min(1, max_norm / (norm + eps)): in place, or into the tensors out.  No tensor\n"
     "overlaps another.  Returns the\n"
     "norm, float32 [1] on the device (no synchronisation).  A norm that is not finite\n"
     "scales nothing and sets DEVERR_NONFINITE in error_word."},
    {"bind", py_bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer() { return PyModule_Create(&module); }
