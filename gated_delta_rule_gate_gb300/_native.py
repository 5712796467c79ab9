"""ctypes view of the C ABI declared in include/gdn.h (libgdn.so).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind these symbols.  There is no CPU fallback; if the library is
missing and cannot be built, loading raises.
"""
import ctypes
import os
import threading

from . import build as _build

GDN_OK, GDN_ERR_INVALID, GDN_ERR_UNSUPPORTED, GDN_ERR_WORKSPACE, GDN_ERR_CUDA = range(5)
DTYPE_F32, DTYPE_F16, DTYPE_BF16, DTYPE_E4M3 = 0, 1, 2, 3
RULES = {"linear": 0, "gated": 1, "delta": 2, "gated_delta": 3, "gdn2": 4}
FLAG_L2NORM_Q, FLAG_L2NORM_K, FLAG_BETA_SIGMOID, FLAG_DECAY_PER_KEY = 0x1, 0x2, 0x4, 0x8
FLAG_BETA_SHARED = 0x10
FLAG_STATE_KMAJOR = 0x20
DEVERR_BAD_SLOT, DEVERR_TIMEOUT, DEVERR_OVERLAP, DEVERR_DECAY_RANGE = 0x1, 0x2, 0x4, 0x8
DEVERR_NONFINITE = 0x10

EXPORTS = ("gdn_gate", "gdn_recurrent_step", "gdn_chunked_prefill_workspace_size",
           "gdn_chunked_prefill_workspace_size_min", "gdn_chunked_prefill", "gdn_chunked_prefill_noalloc",
           "gdn_status_string", "gdn_last_error_message", "gdn_scan", "gdn_scan_step",
           "gdn_scan_backward", "gdn_rmsnorm", "gdn_rmsnorm_backward", "gdn_rmsnorm_backward_workspace_size",
           "gdn_grad_clip", "gdn_grad_clip_workspace_size", "gdn_glu", "gdn_glu_workspace_size", "gdn_glu_backward",
           "gdn_glu_backward_workspace_size", "gdn_adamw")
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4}
ADAMW_BLOCK = 256
INPUT_SCALES = {"none": 0, "lerp": 1, "unit": 2}
SCAN_CHUNK = 64

_vp = ctypes.c_void_p


class GdnProblem(ctypes.Structure):
    """Mirror of ``gdn_problem`` (include/gdn.h)."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("total_tokens", ctypes.c_int32), ("seq_len", ctypes.c_int32),
        ("num_heads_q", ctypes.c_int32), ("num_heads_v", ctypes.c_int32),
        ("head_dim_k", ctypes.c_int32), ("head_dim_v", ctypes.c_int32),
        ("num_state_rows", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
        ("decay_dtype", ctypes.c_int32), ("beta_dtype", ctypes.c_int32),
        ("rule", ctypes.c_int32), ("flags", ctypes.c_uint32), ("scale", ctypes.c_float),
        ("state_update_capacity", ctypes.c_int32),
        ("q", _vp), ("k", _vp), ("v", _vp), ("o", _vp), ("decay", _vp),
        ("gate_bias", _vp), ("gate_scale", _vp), ("beta", _vp),
        ("cu_seqlens", _vp), ("slot_ids", _vp), ("initial_state", _vp),
        ("final_state", _vp), ("error_word", _vp), ("seq_lens", _vp),
        ("erase_gate", _vp), ("write_gate", _vp),
    ]


class GdnGateArgs(ctypes.Structure):
    """Mirror of ``gdn_gate_args`` (include/gdn.h)."""
    _fields_ = [
        ("n", ctypes.c_int64), ("heads", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("a", _vp), ("dt_bias", _vp), ("decay_scale", _vp), ("b", _vp),
        ("decay_out", _vp), ("beta_out", _vp),
    ]


class GdnScanArgs(ctypes.Structure):
    """Mirror of ``gdn_scan_args`` (include/gdn.h)."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("total_tokens", ctypes.c_int32), ("seq_len", ctypes.c_int32),
        ("channels", ctypes.c_int32), ("num_state_rows", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
        ("gate_dtype", ctypes.c_int32), ("input_scale", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("x_stride", ctypes.c_int64), ("decay_stride", ctypes.c_int64), ("beta_stride", ctypes.c_int64),
        ("o_stride", ctypes.c_int64),
        ("x", _vp), ("decay", _vp), ("beta", _vp), ("o", _vp), ("gate_bias", _vp), ("gate_scale", _vp),
        ("cu_seqlens", _vp), ("seq_lens", _vp), ("slot_ids", _vp), ("initial_state", _vp),
        ("final_state", _vp), ("chunk_states", _vp), ("error_word", _vp),
    ]


class GdnScanGradArgs(ctypes.Structure):
    """Mirror of ``gdn_scan_grad_args`` (include/gdn.h)."""
    _fields_ = [
        ("forward", GdnScanArgs),
        ("d_o_stride", ctypes.c_int64), ("dx_stride", ctypes.c_int64), ("d_decay_stride", ctypes.c_int64),
        ("d_beta_stride", ctypes.c_int64),
        ("d_o", _vp), ("d_final_state", _vp), ("dx", _vp), ("d_decay", _vp), ("d_beta", _vp),
        ("d_gate_bias", _vp), ("d_gate_scale", _vp), ("d_initial_state", _vp),
    ]


class GdnRmsnormArgs(ctypes.Structure):
    """Mirror of ``gdn_rmsnorm_args`` (include/gdn.h)."""
    _fields_ = [
        ("rows", ctypes.c_int64), ("dim", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
        ("residual_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
        ("group", ctypes.c_int32), ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64),
        ("x", _vp), ("residual", _vp), ("weight", _vp), ("out", _vp), ("residual_out", _vp), ("scales", _vp),
        ("rstd", _vp),
    ]


class GdnRmsnormGradArgs(ctypes.Structure):
    """Mirror of ``gdn_rmsnorm_grad_args`` (include/gdn.h)."""
    _fields_ = [
        ("rows", ctypes.c_int64), ("dim", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
        ("r_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("d_out_stride", ctypes.c_int64),
        ("d_out", _vp), ("r", _vp), ("weight", _vp), ("rstd", _vp), ("d_residual", _vp), ("dx", _vp),
        ("d_weight", _vp),
    ]


class GdnGradClipArgs(ctypes.Structure):
    """Mirror of ``gdn_grad_clip_args`` (include/gdn.h)."""
    _fields_ = [
        ("count", ctypes.c_int32), ("max_norm", ctypes.c_float), ("eps", ctypes.c_float),
        ("grads", ctypes.POINTER(_vp)), ("outs", ctypes.POINTER(_vp)), ("sizes", ctypes.POINTER(ctypes.c_int64)),
        ("dtypes", ctypes.POINTER(ctypes.c_int32)), ("norm", _vp), ("error_word", _vp),
    ]


class GdnGluArgs(ctypes.Structure):
    """Mirror of ``gdn_glu_args`` (include/gdn.h)."""
    _fields_ = [
        ("rows", ctypes.c_int64), ("dim", ctypes.c_int32), ("inner", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("activation", ctypes.c_int32), ("x_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
        ("x", _vp), ("w_gate", _vp), ("w_up", _vp), ("out", _vp), ("gates", _vp), ("error_word", _vp),
    ]


class GdnGluGradArgs(ctypes.Structure):
    """Mirror of ``gdn_glu_grad_args`` (include/gdn.h)."""
    _fields_ = [
        ("rows", ctypes.c_int64), ("dim", ctypes.c_int32), ("inner", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("activation", ctypes.c_int32), ("x_stride", ctypes.c_int64), ("d_out_stride", ctypes.c_int64),
        ("dx_stride", ctypes.c_int64), ("d_out", _vp), ("x", _vp), ("w_gate", _vp), ("w_up", _vp), ("gates", _vp),
        ("dx", _vp), ("d_w_gate", _vp), ("d_w_up", _vp), ("error_word", _vp),
    ]


class GdnAdamwArgs(ctypes.Structure):
    """Mirror of ``gdn_adamw_args`` (include/gdn.h)."""
    _fields_ = [
        ("count", ctypes.c_int32), ("state_dtype", ctypes.c_int32), ("step", ctypes.c_int64), ("lr", ctypes.c_double),
        ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
        ("weight_decay", ctypes.c_double), ("max_norm", ctypes.c_double), ("norm_eps", ctypes.c_double),
        ("params", ctypes.POINTER(_vp)), ("grads", ctypes.POINTER(_vp)), ("exp_avg", ctypes.POINTER(_vp)),
        ("exp_avg_sq", ctypes.POINTER(_vp)), ("exp_avg_scales", ctypes.POINTER(_vp)),
        ("exp_avg_sq_scales", ctypes.POINTER(_vp)), ("master", ctypes.POINTER(_vp)),
        ("sizes", ctypes.POINTER(ctypes.c_int64)), ("param_dtypes", ctypes.POINTER(ctypes.c_int32)),
        ("grad_dtypes", ctypes.POINTER(ctypes.c_int32)), ("step_device", _vp), ("lr_device", _vp),
        ("grad_norm", _vp), ("error_word", _vp),
    ]


class GdnError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        super().__init__("%s: %s" % (status_string(status), message))


_lib = None
_lock = threading.Lock()


def library_path():
    return _build.LIB


def load():
    """Loads libgdn.so (building it first when out of date and nvcc exists)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not _build.up_to_date():
            try:
                _build.build()
            except RuntimeError:
                if not os.path.exists(_build.LIB):
                    raise
        if not os.path.exists(_build.LIB):
            raise RuntimeError("libgdn.so is missing: build it with gated_delta_rule_gate_gb300.build.build()")
        lib = ctypes.CDLL(_build.LIB)
        lib.gdn_gate.argtypes = [ctypes.POINTER(GdnGateArgs), _vp]
        lib.gdn_gate.restype = ctypes.c_int
        lib.gdn_recurrent_step.argtypes = [ctypes.POINTER(GdnProblem), _vp]
        lib.gdn_recurrent_step.restype = ctypes.c_int
        lib.gdn_chunked_prefill_workspace_size.argtypes = [ctypes.POINTER(GdnProblem), ctypes.c_int32]
        lib.gdn_chunked_prefill_workspace_size.restype = ctypes.c_size_t
        lib.gdn_chunked_prefill_workspace_size_min.argtypes = [ctypes.POINTER(GdnProblem), ctypes.c_int32]
        lib.gdn_chunked_prefill_workspace_size_min.restype = ctypes.c_size_t
        lib.gdn_chunked_prefill.argtypes = [ctypes.POINTER(GdnProblem), ctypes.c_int32, _vp,
                                            ctypes.c_size_t, _vp]
        lib.gdn_chunked_prefill.restype = ctypes.c_int
        lib.gdn_chunked_prefill_noalloc.argtypes = [ctypes.POINTER(GdnProblem), ctypes.c_int32, _vp]
        lib.gdn_chunked_prefill_noalloc.restype = ctypes.c_int
        for name, args in (("gdn_scan", GdnScanArgs), ("gdn_scan_step", GdnScanArgs),
                           ("gdn_scan_backward", GdnScanGradArgs), ("gdn_rmsnorm", GdnRmsnormArgs),
                           ("gdn_adamw", GdnAdamwArgs)):
            getattr(lib, name).argtypes = [ctypes.POINTER(args), _vp]
            getattr(lib, name).restype = ctypes.c_int
        for name, args in (("gdn_rmsnorm_backward", GdnRmsnormGradArgs), ("gdn_grad_clip", GdnGradClipArgs),
                           ("gdn_glu", GdnGluArgs), ("gdn_glu_backward", GdnGluGradArgs)):
            getattr(lib, name).argtypes = [ctypes.POINTER(args), _vp, ctypes.c_size_t, _vp]
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name + "_workspace_size").argtypes = [ctypes.POINTER(args)]
            getattr(lib, name + "_workspace_size").restype = ctypes.c_size_t
        lib.gdn_status_string.argtypes = [ctypes.c_int]
        lib.gdn_status_string.restype = ctypes.c_char_p
        lib.gdn_last_error_message.argtypes = []
        lib.gdn_last_error_message.restype = ctypes.c_char_p
        _lib = lib
        return lib


def status_string(status):
    return load().gdn_status_string(int(status)).decode()


def last_error_message():
    return load().gdn_last_error_message().decode()


def check(status):
    if status != GDN_OK:
        raise GdnError(status, last_error_message())
    return status
