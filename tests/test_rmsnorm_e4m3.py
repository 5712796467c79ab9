"""The 8-bit output of gdn_rmsnorm is the formula's value for value: with the rstd and the
scales that the call returns, y = (r rstd) weight and y / s in fp32 are determined to the
bit, and so is the nearest e4m3 value.  No tolerance."""
import pytest
import torch

import layer_reference as ref

E4M3 = torch.float8_e4m3fn


# widths of whole words, of pairs, of neither, and beyond a row's registers; enough values
# that some lie at the edge of two steps
@pytest.mark.gpu
@pytest.mark.parametrize("n,D", [(2048, 4096), (4000, 518), (4000, 517), (1000, 8200), (600, 8201)])
@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [0, 128])
def test_out_is_y_over_s(n, D, act, group):
    import gated_delta_rule_gate_gb300 as g
    gen = torch.Generator(device="cuda").manual_seed(D + group)
    dt = ref.DT[act]
    x = torch.randn(n, D, generator=gen, device="cuda").to(dt)
    res = (2 * torch.randn(n, D, generator=gen, device="cuda")).to(dt)
    w = (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt)
    got = g.gdn_rmsnorm(x, w, residual=res, out_dtype=E4M3, group=group, want_rstd=True)
    x, res, w, rstd, scales, out = (t.cpu() for t in (x, res, w, got.rstd, got.scales, got.out))
    y = (x.float() + res.float()) * rstd[:, None] * w.float()
    s = scales.view(n, -1).repeat_interleave(group or D, dim=1)[:, :D]
    want = (y / s).clamp(-448, 448).to(E4M3)  # the largest value may round to just above 448
    assert int((out.view(torch.uint8) != want.view(torch.uint8)).sum()) == 0
    peak = torch.stack([p.abs().amax(1) for p in y.split(group or D, dim=1)], 1) / 448
    # the scale of a row is formed of max |r weight|, times rstd: three roundings of fp32 apart
    assert bool(((scales.view(n, -1) - peak).abs() <= 4 * 2.0 ** -24 * peak).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [520, 518, 517, 8201])
@pytest.mark.parametrize("group", [0, 128])
def test_zeros_keep_their_signs(D, group):
    import gated_delta_rule_gate_gb300 as g
    gen = torch.Generator().manual_seed(D)
    x = torch.randn(20, D, generator=gen)
    x[:, ::7] = 0.0
    x[:, 1::7] = -0.0
    x[0] = -0.0  # a whole row
    w = torch.randn(D, generator=gen)
    out = g.gdn_rmsnorm(x.cuda(), w.cuda(), out_dtype=E4M3, group=group).out.cpu()
    zero = x == 0
    want = torch.where(torch.signbit(x) != torch.signbit(w), 128, 0)[zero].to(torch.uint8)
    assert torch.equal(out.view(torch.uint8)[zero], want)
