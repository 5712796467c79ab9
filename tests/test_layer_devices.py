"""Where the tensors of a call may lie."""
import pytest
import torch

from layer_standins import Standin

T, D = 6, 8
X, W = Standin((T, D)), Standin((D,))


def with_workspace(ws):
    import gated_delta_rule_gate_gb300 as g
    return [lambda: g.gdn_rmsnorm_backward(X, X, W, Standin((T,)), workspace=ws),
            lambda: g.gdn_grad_clip([X], 1.0, workspace=ws)]


@pytest.mark.parametrize("i", [0, 1])
def test_workspace_of_the_host_is_refused(i):
    with pytest.raises(ValueError, match="workspace is on cpu"):
        with_workspace(torch.empty(1 << 20, dtype=torch.uint8))[i]()


@pytest.mark.parametrize("i", [0, 1])
def test_workspace_in_pieces_is_refused(i):
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        with_workspace(Standin((1 << 10, 4), (8, 1)))[i]()


@pytest.mark.gpu
def test_given_workspace_is_used():
    import gated_delta_rule_gate_gb300 as g
    gen = torch.Generator().manual_seed(1)
    x, d, w = (torch.randn(*s, generator=gen).cuda() for s in ((40, 96), (40, 96), (96,)))
    rstd = g.gdn_rmsnorm(x, w, want_rstd=True).rstd
    want, norm = g.gdn_rmsnorm_backward(d, x, w, rstd), g.gdn_grad_clip([x.clone(), d.clone()], 1.0)
    for ws in (torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), torch.empty(512, 512, device="cuda")):
        got = g.gdn_rmsnorm_backward(d, x, w, rstd, workspace=ws)
        assert torch.equal(got.dx, want.dx) and torch.equal(got.dweight, want.dweight)
        assert torch.equal(g.gdn_grad_clip([x.clone(), d.clone()], 1.0, workspace=ws), norm)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(g.GdnError, match="workspace needs"):
        g.gdn_rmsnorm_backward(d, x, w, rstd, workspace=small)


OTHER = dict(device="cuda:1")


def mixed():
    """Calls whose tensors lie on cuda:0 but for one."""
    import gated_delta_rule_gate_gb300 as g
    x1, w1 = Standin((T, D), **OTHER), Standin((D,), **OTHER)
    i1 = lambda n: Standin((n,), dtype=torch.int32, **OTHER)
    s1, ch = Standin((1, D), **OTHER), Standin((1, D))
    x3 = Standin((2, 3, D))
    for fn in (g.gdn_scan, g.gdn_scan_step):
        yield lambda fn=fn: fn(X, x1)
        yield lambda fn=fn: fn(X, X, beta=x1)
        yield lambda fn=fn: fn(X, X, gate_bias=w1, gate_scale=W)
        yield lambda fn=fn: fn(X, X, gate_bias=W, gate_scale=w1)
        yield lambda fn=fn: fn(X, X, cu_seqlens=i1(2))
        yield lambda fn=fn: fn(x3, x3, seq_lens=i1(2))
        yield lambda fn=fn: fn(X, X, slot_ids=i1(1))
        yield lambda fn=fn: fn(X, X, initial_state=s1)
        yield lambda fn=fn: fn(X, X, final_state=s1)
        yield lambda fn=fn: fn(X, X, out=x1)
        yield lambda fn=fn: fn(X, X, error_word=i1(1))
    b = g.gdn_scan_backward
    yield lambda: b(x1, X, X, ch)
    yield lambda: b(X, X, x1, ch)
    yield lambda: b(X, X, X, s1)
    yield lambda: b(X, X, X, ch, d_final_state=s1)
    yield lambda: b(X, X, X, ch, initial_state=s1)
    yield lambda: b(X, X, X, ch, dx=x1)
    yield lambda: b(X, X, X, ch, d_decay=x1)
    yield lambda: b(X, X, X, ch, beta=X, d_beta=x1)
    yield lambda: b(X, X, X, ch, gate_bias=W, gate_scale=W, d_gate_bias=w1)
    yield lambda: b(X, X, X, ch, gate_bias=W, gate_scale=W, d_gate_scale=w1)
    yield lambda: b(X, X, X, ch, initial_state=ch, d_initial_state=s1)
    yield lambda: g.gdn_rmsnorm(X, w1)
    yield lambda: g.gdn_rmsnorm(X, W, residual=x1)
    yield lambda: g.gdn_rmsnorm(X, W, out=x1)
    yield lambda: g.gdn_rmsnorm(X, W, residual=X, residual_out=x1)
    yield lambda: g.gdn_rmsnorm(X, W, out_dtype=torch.float8_e4m3fn, scales=Standin((T,), **OTHER))
    n = g.gdn_rmsnorm_backward
    yield lambda: n(x1, X, W, Standin((T,)))
    yield lambda: n(X, X, w1, Standin((T,)))
    yield lambda: n(X, X, W, Standin((T,), **OTHER))
    yield lambda: n(X, X, W, Standin((T,)), d_residual=x1)
    yield lambda: n(X, X, W, Standin((T,)), dx=x1)
    yield lambda: n(X, X, W, Standin((T,)), d_weight=w1)
    yield lambda: n(X, X, W, Standin((T,)), workspace=x1)
    c = g.gdn_grad_clip
    yield lambda: c([X, x1], 1.0)
    yield lambda: c([X], 1.0, out=[x1])
    yield lambda: c([X], 1.0, norm=Standin((1,), **OTHER))
    yield lambda: c([X], 1.0, error_word=i1(1))
    yield lambda: c([X], 1.0, workspace=x1)


@pytest.mark.parametrize("i", range(22 + 11 + 12 + 5))
def test_tensors_of_two_devices_are_refused(i):
    calls = list(mixed())
    assert len(calls) == 50
    with pytest.raises(ValueError, match="is on cuda:1, not on cuda:0"):
        calls[i]()
