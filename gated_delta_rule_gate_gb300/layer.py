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


# The current stream's handle without building a stream object (3 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(stream, t):
    if stream is None:
        if _raw_stream is not None and t.is_cuda:
            return _raw_stream(t.get_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_here = contextlib.nullcontext()


def _on(stream):
    """Memory made inside belongs to the stream that the kernels run on."""
    if stream is None:
        return _here
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _lib():
    return N._lib or N.load()


def _call(status):
    if status:
        N.check(status)


def _dtype(t, what):
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError("%s: unsupported dtype %s" % (what, t.dtype)) from None


def _ptr(t, dtype, what, shape=None):
    """Address of a contiguous device tensor of the given dtype, or None."""
    if t is None:
        return None
    if t.is_cuda and t.dtype is dtype and t.is_contiguous() and (shape is None or t.shape == shape):
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError("libgdn takes device tensors; %s is on %s" % (what, t.device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s" % (what, dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    raise ValueError("%s must be %s, got %s" % (what, tuple(shape), tuple(t.shape)))


def _rows(t, dtype, shape, what):
    """(address, elements between rows) of a device tensor whose last dimension
    is contiguous and whose leading ones lie in it as one."""
    if t is None:
        return None, 0
    if not t.is_cuda:
        raise ValueError("libgdn takes device tensors; %s is on %s" % (what, t.device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s" % (what, dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if t.is_contiguous():
        return t.data_ptr(), shape[-1]
    if t.stride(-1) != 1 and shape[-1] != 1:
        raise ValueError("%s must have contiguous channels" % what)
    step = t.stride(-2) if t.dim() > 1 else shape[-1]
    for d in range(t.dim() - 3, -1, -1):  # the leading dimensions as one
        if shape[d + 1] == 1:
            step = t.stride(d)
        elif shape[d] > 1 and t.stride(d) != shape[d + 1] * t.stride(d + 1):
            raise ValueError("%s must have one stride over all its rows" % what)
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
    scale = N.INPUT_SCALES.get(input_scale)
    if scale is None:
        raise ValueError("input_scale must be one of %s" % ", ".join(N.INPUT_SCALES))
    act_dtype, gate_dtype = x.dtype, decay.dtype
    xp, xs = _rows(x, act_dtype, shape, "x")
    gp, gs = _rows(decay, gate_dtype, shape, "decay")
    bp, bs = _rows(beta, gate_dtype, shape, "beta")
    op, os = _rows(out, act_dtype, shape, "out")
    state = initial_state if initial_state is not None else final_state
    rows, state_shape = 0, None
    if state is not None:
        state_shape = state.shape
        if len(state_shape) != 2 or state_shape[1] != D:
            raise ValueError("states must be [rows, %d]" % D)
        rows = state_shape[0]
    f32, i32 = torch.float32, torch.int32
    return N.GdnScanArgs(
        B, T, seq_len, D, rows, act, gate, scale,
        N.FLAG_BETA_SIGMOID if beta_sigmoid else 0, xs, gs, bs, os, xp, gp, bp, op,
        _ptr(gate_bias, f32, "gate_bias", (D,)), _ptr(gate_scale, f32, "gate_scale", (D,)),
        _ptr(cu_seqlens, i32, "cu_seqlens"), _ptr(seq_lens, i32, "seq_lens", (B,)),
        _ptr(slot_ids, i32, "slot_ids", (B,)), _ptr(initial_state, f32, "initial_state"),
        _ptr(final_state, f32, "final_state", state_shape),
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
    _call(_lib().gdn_scan(args, _handle(stream, x)))
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
    _call(_lib().gdn_scan_step(args, _handle(stream, x)))
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
    forward = _scan_args(x, decay, beta, gate_bias, gate_scale, beta_sigmoid, input_scale, cu_seqlens, seq_lens,
                         slot_ids, like, None, None, chunk_states, error_word)
    if initial_state is None:
        forward.initial_state = None
    shape = x.shape
    dop, dos = _rows(d_out, x.dtype, shape, "d_out")
    dxp, dxs = _rows(dx, x.dtype, shape, "dx")
    dgp, dgs = _rows(d_decay, decay.dtype, shape, "d_decay")
    dbp, dbs = _rows(d_beta, decay.dtype, shape, "d_beta")
    rows = None if like is None else like.shape
    args = N.GdnScanGradArgs(
        forward, dos, dxs, dgs, dbs, dop, _ptr(d_final_state, f32, "d_final_state", rows), dxp, dgp, dbp,
        _ptr(d_gate_bias, f32, "d_gate_bias", (D,)), _ptr(d_gate_scale, f32, "d_gate_scale", (D,)),
        _ptr(d_initial_state, f32, "d_initial_state", rows))
    _call(_lib().gdn_scan_backward(args, _handle(stream, x)))
    return ScanGradients(dx, d_decay, d_beta, d_gate_bias, d_gate_scale, d_initial_state)


def gdn_rmsnorm(x, weight, *, residual=None, eps=1e-6, out_dtype=None, group=0, want_rstd=False, out=None,
                residual_out=None, scales=None, stream=None):
    """r = x + residual; out = r / sqrt(mean(r^2) + eps) * weight over the last
    dimension, in fp32.  ``out_dtype`` is x's, or torch.float8_e4m3fn with fp32 scales
    (out * scale is the value): one per row (``group`` 0) or per 128 columns (128).
    Returns NormResult(out, residual, scales, rstd): residual is r in residual's dtype
    (float32 or x's; ``residual_out`` may be ``residual``), rstd is for
    gdn_rmsnorm_backward; None where there is none or it was not asked for."""
    shape, dtype, device = x.shape, x.dtype, x.device
    D = shape[-1] if shape else 0
    n = x.numel() // D if D else 0
    e4m3 = out_dtype is torch.float8_e4m3fn
    if out_dtype is None:
        out_dtype = dtype
    f32, res = torch.float32, None if residual is None else residual.dtype
    rstd, sshape = None, None
    if e4m3:
        sshape = shape[:-1] if group == 0 else shape[:-1] + (-(-D // 128),)
    with _on(stream):
        if out is None:
            out = torch.empty(shape, dtype=out_dtype, device=device)
        if residual is not None and residual_out is None:
            residual_out = torch.empty(shape, dtype=res, device=device)
        if e4m3 and scales is None:
            scales = torch.empty(sshape, dtype=f32, device=device)
        if want_rstd:
            rstd = torch.empty(shape[:-1], dtype=f32, device=device)
    xp, xs = _rows(x, dtype, shape, "x")
    code = _dtype(x, "x")
    args = N.GdnRmsnormArgs(
        n, D, code, code if residual is None else _dtype(residual, "residual"), _dtype(weight, "weight"),
        N.DTYPE_E4M3 if e4m3 else _DT.get(out_dtype, -1), group, eps, xs, xp,
        _ptr(residual, res, "residual", shape), _ptr(weight, weight.dtype, "weight", (D,)),
        _ptr(out, out_dtype, "out", shape), _ptr(residual_out, res, "residual_out", shape),
        _ptr(scales, f32, "scales", sshape), None if rstd is None else rstd.data_ptr())
    _call(_lib().gdn_rmsnorm(args, _handle(stream, x)))
    return NormResult(out, residual_out if residual is not None else None, scales, rstd)


def gdn_rmsnorm_backward(d_out, r, weight, rstd, *, d_residual=None, dx=None, d_weight=None, workspace=None,
                         stream=None):
    """Gradients of gdn_rmsnorm for the gradient ``d_out`` of its (unquantised)
    output and ``d_residual`` of the residual that it returned; r is that residual (x
    where there was none), rstd what it returned.  Returns NormGradients(dx, dweight): dx, in r's dtype, is the
    gradient of x and of residual alike (``dx`` may be ``d_residual``); dweight is
    float32."""
    shape, dtype, device = r.shape, r.dtype, r.device
    D = shape[-1] if shape else 0
    n = r.numel() // D if D else 0
    f32 = torch.float32
    with _on(stream):
        if dx is None:
            dx = torch.empty(shape, dtype=dtype, device=device)
        if d_weight is None:
            d_weight = torch.empty(D, dtype=f32, device=device)
    dp, ds = _rows(d_out, d_out.dtype, shape, "d_out")
    args = N.GdnRmsnormGradArgs(
        n, D, _dtype(d_out, "d_out"), _dtype(r, "r"), _dtype(weight, "weight"), ds, dp, _ptr(r, dtype, "r"),
        _ptr(weight, weight.dtype, "weight", (D,)), _ptr(rstd, f32, "rstd", shape[:-1]),
        _ptr(d_residual, dtype, "d_residual", shape), _ptr(dx, dtype, "dx", shape),
        _ptr(d_weight, f32, "d_weight", (D,)))
    lib = _lib()
    _with_workspace(lib.gdn_rmsnorm_backward, lib.gdn_rmsnorm_backward_workspace_size, args, workspace, r, stream)
    return NormGradients(dx, d_weight)


_TOO_LARGE = ctypes.c_size_t(-1).value


def _with_workspace(call, size, args, workspace, like, stream):
    if workspace is None:
        need = size(args)
        if need == _TOO_LARGE:
            need = 0  # the call says what is wrong
        with _on(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
    _call(call(args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), _handle(stream, like)))


def gdn_grad_clip(grads, max_norm, *, eps=1e-6, out=None, norm=None, error_word=None, workspace=None, stream=None):
    """The 2-norm of all elements of the tensors ``grads`` together, and each scaled
    by min(1, max_norm / (norm + eps)): in place, or into the tensors ``out``.  Returns
    the norm, float32 [1] on the device (no synchronisation).  A norm that is not
    finite scales nothing and sets DEVERR_NONFINITE in ``error_word``."""
    grads = list(grads)
    count = len(grads)
    f32, outs = torch.float32, None
    types = [t.dtype for t in grads]
    with _on(stream):
        if norm is None:
            norm = torch.empty(1, dtype=f32, device=grads[0].device if count else "cuda")
    table = [_ptr(t, d, "a gradient") for t, d in zip(grads, types)]
    try:
        codes = [_DT[d] for d in types]
    except KeyError as e:
        raise TypeError("a gradient: unsupported dtype %s" % e) from None
    pointers = ctypes.c_void_p * count
    if out is not None:
        out = list(out)
        if len(out) != count:
            raise ValueError("out must have a tensor for each of the %d gradients" % count)
        outs = pointers(*[_ptr(o, d, "an output", t.shape) for o, d, t in zip(out, types, grads)])
    args = N.GdnGradClipArgs(count, max_norm, eps, pointers(*table), outs,
                             (ctypes.c_int64 * count)(*[t.numel() for t in grads]), (ctypes.c_int32 * count)(*codes),
                             _ptr(norm, f32, "norm", (1,)), _ptr(error_word, torch.int32, "error_word"))
    lib = _lib()
    _with_workspace(lib.gdn_grad_clip, lib.gdn_grad_clip_workspace_size, args, workspace, norm, stream)
    return norm
