"""Token counts at the end of the 32-bit range: what the walk along time adds to one has to
stay in it."""
import ctypes

import pytest

from gated_delta_rule_gate_gb300 import _native as N
from test_scan import FAKE

MOST = 2 ** 31 - 1 - 8192


def calls(T):
    f = N.GdnScanArgs(1, T, 0, 1, 0, N.DTYPE_F16, N.DTYPE_F16, 0, 0, 0, 0, 0, 0, FAKE, FAKE, None, FAKE)
    b = N.GdnScanGradArgs(f, 0, 0, 0, 0, FAKE, None, FAKE, FAKE)
    b.forward.chunk_states = FAKE
    lib = N.load()
    return [lambda: lib.gdn_scan(ctypes.byref(f), None), lambda: lib.gdn_scan_backward(ctypes.byref(b), None)]


@pytest.mark.parametrize("T", [MOST + 1, 2 ** 31 - 1])
@pytest.mark.parametrize("i", [0, 1])
def test_more_tokens_are_refused(T, i):
    assert calls(T)[i]() == N.GDN_ERR_UNSUPPORTED
    assert "total_tokens above %d" % MOST in N.last_error_message()
