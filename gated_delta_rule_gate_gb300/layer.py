"""Python binding of the recurrent-layer operators, over torch tensors.

As in the rest of the binding, these functions read shapes, strides, dtypes and
pointers, fill the C structs of include/gdn.h and call the library on the current
stream (or ``stream``); what they allocate when an output is not given is torch
memory of that stream.  float32, float16 and bfloat16 tensors are taken.
"""
import contextlib
import ctypes
from collections import namedtuple

import torch

from . import _native as N

_DT = {torch.float32: N.DTYPE_F32, torch.float16: N.DTYPE_F16, torch.bfloat16: N.DTYPE_BF16}

ScanGradients = namedtuple("ScanGradients", "dx d_decay d_beta d_gate_bias d_gate_scale d_initial_state")

NormResult = namedtuple("NormResult", "out residual scales rstd")
NormGradients = namedtuple("NormGradients", "dx dweight")


def _handle(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on(stream):
    """Memory made inside belongs to the stream that the kernels run on."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _dtype(t, what):
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError("%s: unsupported dtype %s" % (what, t.dtype)) from None


def _ptr(t, dtype, what, shape=None):
    """Address of a contiguous device tensor of the given dtype, or None."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libgdn takes device tensors; %s is on %s" % (what, t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s" % (what, dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    if shape is not None and t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    return t.data_ptr()


def _rows(t, shape, what):
    """(address, elements between rows) of a device tensor whose last dimension
    is contiguous and whose leading ones lie in it as one."""
    if t is None:
        return None, 0
    if not t.is_cuda:
        raise ValueError("libgdn takes device tensors; %s is on %s" % (what, t.device))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if t.is_contiguous():
        return t.data_ptr(), shape[-1]
    if t.stride(-1) != 1 and shape[-1] != 1:
        raise ValueError("%s must have contiguous channels" % what)
    step = t.stride(-2)
    if t.dim() == 3 and shape[0] > 1:
        if shape[1] == 1:
            step = t.stride(0)
        elif t.stride(0) != shape[1] * step:
            raise ValueError("%s must have one stride over all tokens" % what)
    return t.data_ptr(), step


def _scan_args(x, decay, beta, gate_bias, gate_scale, beta_sigmoid, input_scale, cu_seqlens, seq_lens, slot_ids,
               initial_state, final_state, out, chunk_states, error_word):
    shape = x.shape
    dim = len(shape)
    act, gate = _dtype(x, "x"), _dtype(decay, "decay")
    if dim == 2:
        T, D = shape
        seq_len = 0
        B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
        if B < 0:
            raise ValueError("cu_seqlens must have batch + 1 entries")
    elif dim == 3:
        B, seq_len, D = shape
        T = B * seq_len
        if cu_seqlens is not None:
            raise ValueError("cu_seqlens goes with packed tokens, x [tokens, channels]")
    else:
        raise ValueError("x must be [tokens, channels] or [batch, tokens, channels]")
    if input_scale not in N.INPUT_SCALES:
        raise ValueError("input_scale must be one of %s" % ", ".join(N.INPUT_SCALES))
    if beta is not None and beta.dtype != decay.dtype:
        raise TypeError("beta must have the dtype of decay")
    if out is not None and out.dtype != x.dtype:
        raise TypeError("out must have the dtype of x")
    xp, xs = _rows(x, shape, "x")
    gp, gs = _rows(decay, shape, "decay")
    bp, bs = _rows(beta, shape, "beta")
    op, os = _rows(out, shape, "out")
    state = initial_state if initial_state is not None else final_state
    rows = 0
    if state is not None:
        if state.dim() != 2 or state.shape[1] != D:
            raise ValueError("states must be [rows, %d]" % D)
        rows = state.shape[0]
    f32, i32 = torch.float32, torch.int32
    return N.GdnScanArgs(
        B, T, seq_len, D, rows, act, gate, N.INPUT_SCALES[input_scale],
        N.FLAG_BETA_SIGMOID if beta_sigmoid else 0, xs, gs, bs, os, xp, gp, bp, op,
        _ptr(gate_bias, f32, "gate_bias", (D,)), _ptr(gate_scale, f32, "gate_scale", (D,)),
        _ptr(cu_seqlens, i32, "cu_seqlens"), _ptr(seq_lens, i32, "seq_lens", (B,)),
        _ptr(slot_ids, i32, "slot_ids", (B,)), _ptr(initial_state, f32, "initial_state"),
        _ptr(final_state, f32, "final_state", None if state is None else state.shape),
        _ptr(chunk_states, f32, "chunk_states", (-(-T // N.SCAN_CHUNK), D)), _ptr(error_word, i32, "error_word"))


def gdn_scan(x, decay, *, beta=None, gate_bias=None, gate_scale=None, beta_sigmoid=False, input_scale="none",
             cu_seqlens=None, seq_lens=None, slot_ids=None, initial_state=None, final_state=None, out=None,
             want_chunk_states=False, error_word=None, stream=None):
    """The gated linear recurrence over whole sequences, per channel

        g = decay, or gate_scale * softplus(decay + gate_bias);  a = exp(g)
        h_t = a h_{t-1} + n i x_t;  out_t = h_t

    with i = 1, ``beta`` or sigmoid(``beta``) and n = 1, 1 - a ("lerp") or
    sqrt(1 - a^2) ("unit").  x, decay and beta are [T, D] packed (requests by
    ``cu_seqlens``, else one) or [B, S, D] (``seq_lens`` bounds the rows); they may
    be columns of wider tensors.  States are fp32 [rows, D], row ``slot_ids[b]`` or
    b; ``final_state`` is written if given and may be ``initial_state``.  Returns
    out (allocated when not given; tokens of no request are not written), or (out,
    chunk_states) with ``want_chunk_states``, for gdn_scan_backward."""
    chunks = None
    if out is None or want_chunk_states:
        with _on(stream):
            if out is None:
                out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            if want_chunk_states:
                D = x.shape[-1]
                chunks = torch.empty(-(-x.numel() // max(D, 1) // N.SCAN_CHUNK), D, device=x.device)
    args = _scan_args(x, decay, beta, gate_bias, gate_scale, beta_sigmoid, input_scale, cu_seqlens, seq_lens,
                      slot_ids, initial_state, final_state, out, chunks, error_word)
    N.check(N.load().gdn_scan(args, _handle(stream)))
    return (out, chunks) if want_chunk_states else out


def gdn_scan_step(x, decay, *, beta=None, gate_bias=None, gate_scale=None, beta_sigmoid=False, input_scale="none",
                  cu_seqlens=None, seq_lens=None, slot_ids=None, initial_state=None, final_state=None, out=None,
                  error_word=None, stream=None):
    """gdn_scan for one or a few tokens a request (time grows with the longest):
    the serving step, usually with ``initial_state`` and ``final_state`` one slab
    that ``slot_ids`` address."""
    if out is None:
        with _on(stream):
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    args = _scan_args(x, decay, beta, gate_bias, gate_scale, beta_sigmoid, input_scale, cu_seqlens, seq_lens,
                      slot_ids, initial_state, final_state, out, None, error_word)
    N.check(N.load().gdn_scan_step(args, _handle(stream)))
    return out


def gdn_scan_backward(d_out, x, decay, chunk_states, *, beta=None, gate_bias=None, gate_scale=None,
                      beta_sigmoid=False, input_scale="none", cu_seqlens=None, seq_lens=None, slot_ids=None,
                      initial_state=None, d_final_state=None, dx=None, d_decay=None, d_beta=None, d_gate_bias=None,
                      d_gate_scale=None, d_initial_state=None, error_word=None, stream=None):
    """Gradients of gdn_scan for the gradient ``d_out`` of its output (and
    ``d_final_state`` of its final states): the forward call's arguments and the
    chunk_states that it returned.  Returns ScanGradients(dx, d_decay, d_beta,
    d_gate_bias, d_gate_scale, d_initial_state), None where there is no such input.
    Outputs are allocated when not given (zeros where tokens or state rows may belong
    to no request); a given one is not written there."""
    like = initial_state if initial_state is not None else d_final_state
    # every token and row is written unless requests may leave some out
    token = torch.empty_like if cu_seqlens is None and seq_lens is None and slot_ids is None else torch.zeros_like
    with _on(stream):
        if dx is None:
            dx = token(x, memory_format=torch.contiguous_format)
        if d_decay is None:
            d_decay = token(decay, memory_format=torch.contiguous_format)
        if d_beta is None and beta is not None:
            d_beta = token(beta, memory_format=torch.contiguous_format)
        if gate_bias is not None:
            if d_gate_bias is None:
                d_gate_bias = torch.empty_like(gate_bias)
            if d_gate_scale is None:
                d_gate_scale = torch.empty_like(gate_scale)
        if d_initial_state is None and initial_state is not None:
            d_initial_state = torch.zeros_like(initial_state)
    f32, D = torch.float32, x.shape[-1]
    for t, of, what in ((d_out, x, "d_out"), (dx, x, "dx"), (d_decay, decay, "d_decay"), (d_beta, beta, "d_beta")):
        if t is not None and of is not None and t.dtype != of.dtype:
            raise TypeError("%s must be %s" % (what, of.dtype))
    forward = _scan_args(x, decay, beta, gate_bias, gate_scale, beta_sigmoid, input_scale, cu_seqlens, seq_lens,
                         slot_ids, like, None, None, chunk_states, error_word)
    if initial_state is None:
        forward.initial_state = None
    dop, dos = _rows(d_out, x.shape, "d_out")
    dxp, dxs = _rows(dx, x.shape, "dx")
    dgp, dgs = _rows(d_decay, x.shape, "d_decay")
    dbp, dbs = _rows(d_beta, x.shape, "d_beta")
    rows = None if like is None else like.shape
    args = N.GdnScanGradArgs(
        forward, dos, dxs, dgs, dbs, dop, _ptr(d_final_state, f32, "d_final_state", rows), dxp, dgp, dbp,
        _ptr(d_gate_bias, f32, "d_gate_bias", (D,)), _ptr(d_gate_scale, f32, "d_gate_scale", (D,)),
        _ptr(d_initial_state, f32, "d_initial_state", rows))
    N.check(N.load().gdn_scan_backward(args, _handle(stream)))
    return ScanGradients(dx, d_decay, d_beta, d_gate_bias, d_gate_scale, d_initial_state)


def gdn_rmsnorm(x, weight, *, residual=None, eps=1e-6, out_dtype=None, group=0, want_rstd=False, out=None,
                residual_out=None, scales=None, stream=None):
    """r = x + residual; out = r / sqrt(mean(r^2) + eps) * weight over the last
    dimension, in fp32.  ``out_dtype`` is x's, or torch.float8_e4m3fn with fp32 scales
    (out * scale is the value): one per row (``group`` 0) or per 128 columns (128).
    Returns NormResult(out, residual, scales, rstd): residual is r in residual's dtype
    (float32 or x's; ``residual_out`` may be ``residual``), rstd is for
    gdn_rmsnorm_backward; None where there is none or it was not asked for."""
    shape = x.shape
    D = shape[-1] if x.dim() else 0
    n = x.numel() // D if D else 0
    e4m3 = out_dtype is torch.float8_e4m3fn
    if out_dtype is None:
        out_dtype = x.dtype
    rstd = None
    with _on(stream):
        if out is None:
            out = torch.empty(shape, dtype=out_dtype, device=x.device)
        if residual is not None and residual_out is None:
            residual_out = torch.empty(shape, dtype=residual.dtype, device=x.device)
        if e4m3 and scales is None:
            cols = () if group == 0 else (-(-D // 128),)
            scales = torch.empty(shape[:-1] + cols, device=x.device)
        if want_rstd:
            rstd = torch.empty(shape[:-1], device=x.device)
    xp, xs = _rows(x, shape, "x")
    res = None if residual is None else residual.dtype
    code = _dtype(x, "x")
    args = N.GdnRmsnormArgs(
        n, D, code, code if residual is None else _dtype(residual, "residual"), _dtype(weight, "weight"),
        N.DTYPE_E4M3 if e4m3 else _DT.get(out_dtype, -1), group, eps, xs, xp,
        _ptr(residual, res, "residual", shape), _ptr(weight, weight.dtype, "weight", (D,)),
        _ptr(out, out_dtype, "out", shape), _ptr(residual_out, res, "residual_out", shape),
        _ptr(scales, torch.float32, "scales", shape[:-1] + (() if group == 0 else (-(-D // 128),))),
        _ptr(rstd, torch.float32, "rstd"))
    N.check(N.load().gdn_rmsnorm(args, _handle(stream)))
    return NormResult(out, residual_out if residual is not None else None, scales, rstd)


def gdn_rmsnorm_backward(d_out, r, weight, rstd, *, d_residual=None, dx=None, d_weight=None, workspace=None,
                         stream=None):
    """Gradients of gdn_rmsnorm for the gradient ``d_out`` of its (unquantised)
    output and ``d_residual`` of the residual that it returned; r is that residual (x
    where there was none), rstd what it returned.  Returns NormGradients(dx, dweight): dx, in r's dtype, is the
    gradient of x and of residual alike (``dx`` may be ``d_residual``); dweight is
    float32."""
    shape = r.shape
    D = shape[-1] if r.dim() else 0
    n = r.numel() // D if D else 0
    with _on(stream):
        if dx is None:
            dx = torch.empty(shape, dtype=r.dtype, device=r.device)
        if d_weight is None:
            d_weight = torch.empty(D, device=r.device)
    dp, ds = _rows(d_out, shape, "d_out")
    args = N.GdnRmsnormGradArgs(
        n, D, _dtype(d_out, "d_out"), _dtype(r, "r"), _dtype(weight, "weight"), ds, dp, _ptr(r, r.dtype, "r"),
        _ptr(weight, weight.dtype, "weight", (D,)), _ptr(rstd, torch.float32, "rstd", shape[:-1]),
        _ptr(d_residual, r.dtype, "d_residual", shape), _ptr(dx, r.dtype, "dx", shape),
        _ptr(d_weight, torch.float32, "d_weight", (D,)))
    _with_workspace("gdn_rmsnorm_backward", args, workspace, r.device, stream)
    return NormGradients(dx, d_weight)


def _with_workspace(name, args, workspace, device, stream):
    lib = N.load()
    if workspace is None:
        need = getattr(lib, name + "_workspace_size")(args)
        if need == ctypes.c_size_t(-1).value:
            need = 0  # the call says what is wrong
        with _on(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
    N.check(getattr(lib, name)(args, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                               _handle(stream)))


def gdn_grad_clip(grads, max_norm, *, eps=1e-6, out=None, norm=None, error_word=None, workspace=None, stream=None):
    """The 2-norm of all elements of the tensors ``grads`` together, and each scaled
    by min(1, max_norm / (norm + eps)): in place, or into the tensors ``out``.  Returns
    the norm, float32 [1] on the device (no synchronisation).  A norm that is not
    finite scales nothing and sets DEVERR_NONFINITE in ``error_word``."""
    grads = list(grads)
    count = len(grads)
    device = grads[0].device if count else torch.device("cuda", torch.cuda.current_device())
    with _on(stream):
        if norm is None:
            norm = torch.empty(1, device=device)
    table = (ctypes.c_void_p * count)()
    sizes = (ctypes.c_int64 * count)()
    types = (ctypes.c_int32 * count)()
    outs = None
    for i, t in enumerate(grads):
        table[i], sizes[i], types[i] = _ptr(t, t.dtype, "a gradient"), t.numel(), _dtype(t, "a gradient")
    if out is not None:
        out = list(out)
        if len(out) != count:
            raise ValueError("out must have a tensor for each of the %d gradients" % count)
        outs = (ctypes.c_void_p * count)()
        for i, t in enumerate(out):
            outs[i] = _ptr(t, grads[i].dtype, "an output", grads[i].shape)
    args = N.GdnGradClipArgs(count, max_norm, eps, table, outs, sizes, types, _ptr(norm, torch.float32, "norm", (1,)),
                             _ptr(error_word, torch.int32, "error_word"))
    _with_workspace("gdn_grad_clip", args, workspace, device, stream)
    return norm
