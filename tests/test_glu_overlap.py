"""gdn_glu and gdn_glu_backward refuse results that lie on what the kernels read meanwhile, or on
one another, and take rows that lie beside one another in one tensor."""
import ctypes

import pytest
import torch

import test_glu as glu
from gated_delta_rule_gate_gb300 import _native as N

AT = 0x10000000  # of operands 16 MB apart
MB = 1 << 20


def addresses(a, names, **over):
    for i, f in enumerate(names):
        setattr(a, f, over.pop(f, AT + 16 * MB * i))
    for k, v in over.items():
        setattr(a, k, v)
    return a


def forward(**over):
    a = glu._forward()
    return addresses(a, ("x", "w_gate", "w_up", "out", "gates"), **over)


def backward(**over):
    a = glu._backward()
    return addresses(a, ("x", "w_gate", "w_up", "d_out", "gates", "dx", "d_w_gate", "d_w_up"), **over)


@pytest.mark.parametrize("over,msg", [
    (dict(out=AT), "out overlaps x"),
    (dict(out=AT + 40 * 24 * 2 - 16), "out overlaps x"),
    (dict(out=AT + 16 * MB - 16), "out overlaps w_gate"),
    (dict(out=AT + 32 * MB + 16 * 24 * 2 - 2), "out overlaps w_up"),
    (dict(gates=AT), "gates overlaps x"),
    (dict(gates=AT + 48 * MB), "out overlaps gates"),
    (dict(out=AT, x_stride=1 << 62), "out overlaps x"),
    (dict(out=AT, out_stride=(1 << 63) - 8), "out overlaps x"),
    # columns of one tensor that have one in common
    (dict(x_stride=48, out=AT + 23 * 2, out_stride=48), "out overlaps x"),
    # rows at unequal distances: the first row of out lies in the second of x
    (dict(x_stride=32, out=AT + 24 * 2, out_stride=48), "out overlaps x"),
])
@pytest.mark.parametrize("rows", [40, 20])
def test_forward_refuses_overlap(over, msg, rows):
    lib, a = N.load(), forward(rows=rows, **over)
    if rows == 20 and over.get("out") == AT + 40 * 24 * 2 - 16:
        a.out = AT + 20 * 24 * 2 - 16
    need = lib.gdn_glu_workspace_size(ctypes.byref(a))
    assert lib.gdn_glu(ctypes.byref(a), 1 << 20, need, None) == N.GDN_ERR_INVALID
    assert msg in N.last_error_message()


@pytest.mark.parametrize("over,msg", [
    (dict(dx=AT), "dx overlaps x"),
    (dict(dx=AT + 16 * MB), "dx overlaps w_gate"),
    (dict(d_w_gate=AT + 20 * 24 * 2 - 2), "d_w_gate overlaps x"),
    (dict(d_w_up=AT + 32 * MB), "d_w_up overlaps w_up"),
    (dict(d_w_up=AT + 96 * MB + 2), "d_w_gate overlaps d_w_up"),
    (dict(d_w_gate=AT + 80 * MB), "dx overlaps d_w_gate"),
    (dict(d_w_gate=AT, dx=None), "d_w_gate overlaps x"),
])
def test_backward_refuses_overlap(over, msg):
    lib, a = N.load(), backward(**over)
    need = lib.gdn_glu_backward_workspace_size(ctypes.byref(a))
    assert lib.gdn_glu_backward(ctypes.byref(a), 1 << 20, need, None) == N.GDN_ERR_INVALID
    assert msg in N.last_error_message()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 70])
def test_rows_beside_one_another(T):
    """x, out, d_out and dx as columns of one tensor; dx in the place of d_out, which has been read by then."""
    import gated_delta_rule_gate_gb300 as gdn
    D, F = 64, 40
    x, wg, wu, d = glu.draw(T, D, F, "bf16", seed=T)
    out, gates = gdn.gdn_glu(x, wg, wu, want_gates=True)
    want = gdn.gdn_glu_backward(d, x, wg, wu, gates)
    for gap in (0, 3):  # whole words and not
        wide = torch.full((T, 2 * (D + F) + 3 * gap), 7.0, dtype=x.dtype, device="cuda")
        at, parts = 0, []
        for n in (D, F, F, D):
            parts.append(wide[:, at:at + n])
            at += n + gap
        xs, outs, ds, dxs = parts
        xs.copy_(x), ds.copy_(d)
        assert torch.equal(gdn.gdn_glu(xs, wg, wu, out=outs), out)
        got = gdn.gdn_glu_backward(ds, xs, wg, wu, gates, dx=dxs)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(xs, x) and torch.equal(ds, d) and torch.equal(outs, out)
        with pytest.raises(gdn.GdnError, match="out overlaps x"):
            gdn.gdn_glu(xs, wg, wu, out=wide[:, 1:1 + F])
        assert torch.equal(xs, x)
    square = torch.randn(T, D, device="cuda").to(x.dtype)
    w2 = [torch.randn(D, D, device="cuda").to(x.dtype) for _ in range(2)]
    _, gates = gdn.gdn_glu(x, *w2, want_gates=True)
    want = gdn.gdn_glu_backward(square, x, *w2, gates)
    got = gdn.gdn_glu_backward(square, x, *w2, gates, dx=square)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(gdn.GdnError, match="dx overlaps x"):
        gdn.gdn_glu_backward(d, x, wg, wu, gdn.gdn_glu(x, wg, wu, want_gates=True)[1], dx=x)
