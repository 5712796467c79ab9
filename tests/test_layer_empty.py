"""Calls with nothing in them: no requests, no tokens."""
import ctypes

import pytest
import torch

from gated_delta_rule_gate_gb300 import _native as N
from layer_standins import Standin


@pytest.mark.gpu
@pytest.mark.parametrize("states", [False, True])
def test_gradient_of_no_requests(states):
    """Offsets of one entry beside tokens: no token belongs to a request, and the sums are zero."""
    import gated_delta_rule_gate_gb300 as g
    for T, D in ((130, 70), (1, 64), (0, 16)):
        x, z, d, b = (torch.randn(T, D, device="cuda") for _ in range(4))
        bias = torch.randn(D, device="cuda")
        # what lies behind the one offset would be a request of all tokens
        cu = torch.tensor([0, T, T], dtype=torch.int32, device="cuda")[:1]
        h = torch.randn(3, D, device="cuda") if states else None
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = dict(beta=b, gate_bias=bias, gate_scale=-bias.exp(), cu_seqlens=cu, initial_state=h, error_word=err)
        _, chunks = g.gdn_scan(x, z, want_chunk_states=True, **kw)
        got = g.gdn_scan_backward(d, x, z, chunks, d_final_state=h, **kw)
        torch.cuda.synchronize()
        for t in got:
            assert t is None or not bool(t.any())
        assert int(err) == 0


@pytest.mark.gpu
def test_gradient_of_no_requests_through_the_library():
    """Without offsets, and without the tensors that no token needs."""
    dbias, dscale, bias = (torch.full((16,), 7.0, device="cuda") for _ in range(3))
    f = N.GdnScanArgs(0, 8, 0, 16, 0, N.DTYPE_F32, N.DTYPE_F32, 0, 0)
    f.gate_bias = f.gate_scale = bias.data_ptr()
    a = N.GdnScanGradArgs(f)
    a.d_gate_bias, a.d_gate_scale = dbias.data_ptr(), dscale.data_ptr()
    assert N.load().gdn_scan_backward(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == N.GDN_OK
    torch.cuda.synchronize()
    assert not bool(dbias.any()) and not bool(dscale.any())


def test_states_of_no_rows_are_refused():
    """Zero rows are the library's word for a row a request."""
    import gated_delta_rule_gate_gb300 as g
    x, none, ch = Standin((4, 8)), Standin((0, 8)), Standin((1, 8))
    for call in (lambda: g.gdn_scan(x, x, initial_state=none), lambda: g.gdn_scan_step(x, x, final_state=none),
                 lambda: g.gdn_scan_backward(x, x, x, ch, initial_state=none),
                 lambda: g.gdn_scan_backward(x, x, x, ch, d_final_state=none),
                 lambda: g.gdn_scan_backward(x, x, x, ch, dx=x, d_decay=x, d_initial_state=none)):
        with pytest.raises(ValueError, match="no rows"):
            call()


@pytest.mark.gpu
def test_padded_rows_of_no_tokens():
    """[B, 0, D] with seq_lens: every request is empty and hands its state on."""
    import gated_delta_rule_gate_gb300 as g
    x = torch.empty(3, 0, 20, device="cuda")
    bias = torch.randn(20, device="cuda")
    h = torch.randn(5, 20, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for seq_lens in (None, i32([0, 4, -1])):
        kw = dict(gate_bias=bias, gate_scale=-bias.exp(), seq_lens=seq_lens, slot_ids=i32([4, 0, 2]))
        for fn in (g.gdn_scan, g.gdn_scan_step):
            fin = torch.full_like(h, 7.0)
            assert fn(x, x, initial_state=h, final_state=fin, **kw).shape == x.shape
            assert torch.equal(fin[[4, 0, 2]], h[[4, 0, 2]]) and bool((fin[[1, 3]] == 7.0).all())
        chunks = torch.empty(0, 20, device="cuda")
        got = g.gdn_scan_backward(x, x, x, chunks, initial_state=h, d_final_state=h, **kw)
        assert torch.equal(got.d_initial_state[[4, 0, 2]], h[[4, 0, 2]])
        assert not bool(got.d_gate_bias.any()) and not bool(got.d_gate_scale.any()) and got.dx.shape == x.shape
