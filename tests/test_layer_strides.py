"""Strides of the rows that the recurrent-layer operators take: rows that overlap (expanded
tensors) are refused, by every argument that may have strides."""
import pytest
import torch

from layer_standins import Standin

T, D = 6, 8
X = Standin((T, D))
W = Standin((D,))
OVER = Standin((T, D), (0, 1))  # one row, expanded
NEAR = Standin((T, D), (D - 1, 1))  # rows that share an element
CHUNKS = Standin((1, D))
RSTD = Standin((T,))


def calls():
    import gated_delta_rule_gate_gb300 as g
    three = lambda t: Standin((2, 3, D), (0, 0, 1)) if t is OVER else Standin((2, 3, D), (3 * (D - 1), D - 1, 1))
    x3 = Standin((2, 3, D))
    for fn in (g.gdn_scan, g.gdn_scan_step):
        yield lambda t, fn=fn: fn(t, X)
        yield lambda t, fn=fn: fn(X, t)
        yield lambda t, fn=fn: fn(X, X, beta=t)
        yield lambda t, fn=fn: fn(X, X, out=t)
        yield lambda t, fn=fn: fn(x3, three(t))
        # one token a request, expanded over the requests
        yield lambda t, fn=fn: fn(Standin((T, 1, D)), Standin((T, 1, D), (t.stride(0), D, 1)))
    b = g.gdn_scan_backward
    yield lambda t: b(t, X, X, CHUNKS)
    yield lambda t: b(X, t, X, CHUNKS)
    yield lambda t: b(X, X, t, CHUNKS)
    yield lambda t: b(X, X, X, CHUNKS, beta=t)
    yield lambda t: b(X, X, X, CHUNKS, dx=t)
    yield lambda t: b(X, X, X, CHUNKS, d_decay=t)
    yield lambda t: b(X, X, X, CHUNKS, beta=X, d_beta=t)
    yield lambda t: g.gdn_rmsnorm(t, W)
    yield lambda t: g.gdn_rmsnorm(three(t), W)
    yield lambda t: g.gdn_rmsnorm_backward(t, X, W, RSTD)


@pytest.mark.parametrize("t", [OVER, NEAR], ids=["expanded", "overlapping"])
@pytest.mark.parametrize("i", range(22))
def test_rows_that_overlap_are_refused(i, t):
    with pytest.raises(ValueError, match="overlap"):
        list(calls())[i](t)


def test_every_call_is_listed():
    assert len(list(calls())) == 22


@pytest.mark.gpu
def test_an_expanded_gradient_is_refused_and_its_copy_taken():
    """What autograd hands back through a sum over the rows."""
    import gated_delta_rule_gate_gb300 as g
    gen = torch.Generator().manual_seed(3)
    x, w, d = (torch.randn(*s, generator=gen).cuda() for s in ((50, 24), (24,), (24,)))
    n = g.gdn_rmsnorm(x, w, want_rstd=True)
    d_out = d.expand(50, 24)
    with pytest.raises(ValueError, match="overlap"):
        g.gdn_rmsnorm_backward(d_out, x, w, n.rstd)
    got = g.gdn_rmsnorm_backward(d_out.contiguous(), x, w, n.rstd)
    x6, w6 = x.double().requires_grad_(), w.double().requires_grad_()
    y = x6 * (x6.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w6
    (y.sum(0) * d.double()).sum().backward()
    for a, b in ((got.dx, x6.grad), (got.dweight, w6.grad)):
        assert float((a.double() - b).abs().max() / b.abs().max()) <= 1e-5
    decay = -torch.rand(24, generator=gen).cuda()
    with pytest.raises(ValueError, match="overlap"):
        g.gdn_scan(x, decay.expand(50, 24))
    out = g.gdn_scan(x, decay.expand(50, 24).contiguous())
    h = torch.zeros(24, dtype=torch.double, device="cuda")
    for t in range(50):
        h = decay.double().exp() * h + x[t].double()
    assert float((out[-1].double() - h).abs().max() / h.abs().max()) <= 1e-5
