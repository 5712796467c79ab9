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
