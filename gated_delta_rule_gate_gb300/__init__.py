"""Gated delta rule recurrence on GB300 (sm_103a): a C-ABI CUDA library
(libgdn.so, declared in include/gdn.h) and a thin torch binding.

Entry points (same names as the C ABI):
    gdn_gate, gdn_recurrent_step, gdn_chunked_prefill,
    gdn_chunked_prefill_workspace_size, gdn_chunked_prefill_workspace_size_min,
    gdn_chunked_prefill_noalloc, gdn_status_string
Recurrent-layer operators:
    gdn_scan, gdn_scan_step, gdn_scan_backward, gdn_rmsnorm, gdn_rmsnorm_backward, gdn_glu,
    gdn_glu_backward, gdn_grad_clip, gdn_adamw
"""
from ._native import GdnError, library_path, load  # noqa: F401
from .api import (gdn_chunked_prefill, gdn_chunked_prefill_noalloc,  # noqa: F401
                  gdn_chunked_prefill_workspace_size, gdn_chunked_prefill_workspace_size_min, gdn_gate,
                  gdn_recurrent_step,
                  gdn_status_string, make_problem)
from .layer import OPERATORS as _LAYER, GluGradients, NormGradients, NormResult, ScanGradients  # noqa: F401


def __getattr__(name):
    """The recurrent-layer operators, loaded at their first use."""
    if name in _LAYER:
        from . import layer
        globals()[name] = getattr(layer, name)
        return globals()[name]
    raise AttributeError("module %r has no attribute %r" % (__name__, name))
