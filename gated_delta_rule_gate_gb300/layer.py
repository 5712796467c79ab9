"""The recurrent-layer operators: gdn_scan, gdn_scan_step, gdn_scan_backward,
gdn_rmsnorm, gdn_rmsnorm_backward, gdn_glu, gdn_glu_backward, gdn_grad_clip, gdn_adamw
(documented in their docstrings).

Their Python entry points are native (csrc/layer_binding.cpp), because a decode step
is over in the time that Python takes to look at its tensors.  The module is built (by g++,
against the installed torch) and loaded at the first use of a name; the library and the
other entry points do without it.

The calls record nothing for autograd: results are plain tensors, whatever the inputs
require.  examples/recurrent_layer.py wraps forward and gradient calls in
torch.autograd.Function.
"""
import ctypes
import importlib.machinery
import importlib.util
import threading
from collections import namedtuple

from . import _native as N
from . import build as _build

ScanGradients = namedtuple("ScanGradients", "dx d_decay d_beta d_gate_bias d_gate_scale d_initial_state")
NormResult = namedtuple("NormResult", "out residual scales rstd")
NormGradients = namedtuple("NormGradients", "dx dweight")
GluGradients = namedtuple("GluGradients", "dx d_w_gate d_w_up")

OPERATORS = ("gdn_scan", "gdn_scan_step", "gdn_scan_backward", "gdn_rmsnorm", "gdn_rmsnorm_backward", "gdn_grad_clip",
             "gdn_glu", "gdn_glu_backward", "gdn_adamw")
# what the module calls, in the order that its bind() takes
_FUNCTIONS = ("gdn_scan", "gdn_scan_step", "gdn_scan_backward", "gdn_rmsnorm", "gdn_rmsnorm_backward",
              "gdn_rmsnorm_backward_workspace_size", "gdn_grad_clip", "gdn_grad_clip_workspace_size", "gdn_glu",
              "gdn_glu_workspace_size", "gdn_glu_backward", "gdn_glu_backward_workspace_size", "gdn_adamw")

_module = None
_lock = threading.Lock()


def load():
    """The native module, built first when out of date, on the loaded library."""
    global _module
    with _lock:
        if _module is None:
            import torch  # noqa: F401  (the module's symbols come from it)
            lib = N.load()
            _build.build_binding()  # one of another torch is not loaded
            name = __package__ + "._layer"
            loader = importlib.machinery.ExtensionFileLoader(name, _build.BINDING)
            spec = importlib.util.spec_from_file_location(name, _build.BINDING, loader=loader)
            module = importlib.util.module_from_spec(spec)
            loader.exec_module(module)
            module.bind(tuple(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in _FUNCTIONS), N.check,
                        ScanGradients, NormResult, NormGradients, GluGradients)
            _module = module
        return _module


def __getattr__(name):
    if name in OPERATORS:
        return getattr(load(), name)
    raise AttributeError("module %r has no attribute %r" % (__name__, name))
