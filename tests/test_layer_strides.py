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


def lead_steps(lead, width):
    """Strides of [*lead, D] columns of a wider contiguous tensor [*lead, width]."""
    strides, step = [], width
    for n in reversed(lead):
        strides.insert(0, step)
        step *= n
    return tuple(strides)


@pytest.mark.parametrize("lead", [(2, 1, 3), (2, 3, 1), (1, 2, 3), (2, 1, 1), (2, 1, 3, 1, 2), (1, 1, 3)])
def test_leading_dimensions_of_one_are_passed_over(lead):
    """Rows in one step are accepted wherever a dimension of one stands and whatever its
    stride, and rows that are not in one are refused."""
    import gated_delta_rule_gate_gb300 as g
    strides = lead_steps(lead, D + 4)
    odd = tuple(12345 if n == 1 else s for n, s in zip(lead, strides))
    for st in (strides, odd):
        with pytest.raises(Exception) as e:  # past the checks of strides, at the missing device
            g.gdn_rmsnorm(Standin((*lead, D), (*st, 1)), W, out_dtype=torch.float16, scales=X)
        assert "stride" not in str(e.value) and "overlap" not in str(e.value)
    wide = [k for k, n in enumerate(lead) if n > 1]
    if len(wide) > 1:
        bad = list(strides)
        bad[wide[0]] += D + 4
        with pytest.raises(ValueError, match="one stride"):
            g.gdn_rmsnorm(Standin((*lead, D), (*bad, 1)), W)


@pytest.mark.gpu
@pytest.mark.parametrize("lead", [(2, 1, 3), (4, 1, 5, 1, 2), (1, 3, 1), (3, 1, 1)])
def test_columns_of_a_wider_tensor_with_dimensions_of_one(lead):
    import gated_delta_rule_gate_gb300 as g
    wide = torch.randn(*lead, 40, generator=torch.Generator().manual_seed(7)).cuda()
    w = torch.ones(24, device="cuda")
    x = wide[..., 8:32]
    f, whole = g.gdn_rmsnorm(x, w, want_rstd=True), g.gdn_rmsnorm(x.contiguous(), w, want_rstd=True)
    assert torch.equal(f.out, whole.out) and torch.equal(f.rstd, whole.rstd)
    b = g.gdn_rmsnorm_backward(x, x.contiguous(), w, f.rstd)
    want = g.gdn_rmsnorm_backward(x.contiguous(), x.contiguous(), w, f.rstd)
    assert torch.equal(b.dx, want.dx) and torch.equal(b.dweight, want.dweight)
