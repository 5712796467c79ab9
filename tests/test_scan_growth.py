"""Gates above 0: a run of tokens may grow by more than fp32 holds while the states in it are
zero, or small, and stay numbers.  Against the token loop in 64 bits, value for value, and
all terms of one sign.

Tolerance.  The factor of a run is good to (4 + 1.25 |g|) 2^-24 of itself for the sum g of
its tokens' (below 300 here) and rounded some 40 times on the way (8 warps and 16 blocks,
folded twice); windows follow one another some 16 times at most: under 1e-3 of a state."""
import pytest
import torch

import layer_reference as ref

TOL = 1e-3


def patterns():
    up = lambda n, g: torch.full((n,), g)
    return {
        "steady": up(130, 1.0),
        "steep": torch.cat([up(60, -0.2), up(65, 2.0), up(9, -0.2)]),
        "steep and down": torch.cat([up(50, 2.5), up(50, -2.5), up(50, 2.5), up(40, -2.5)]),
        "slow": up(700, 0.15),
        "in a few tokens": torch.cat([up(40, -0.1), up(16, 6.0), up(60, 0.0)]),
        "up and down": torch.cat([up(100, 1.0), up(100, -1.0), up(100, 1.0), up(90, -1.0)]),
        "down and up": torch.cat([up(70, -0.5), up(150, 0.8), up(30, 0.0)]),
        "far beyond": up(2000, 1.0),
    }


def run(p, d_out, fns):
    import gated_delta_rule_gate_gb300 as g
    c = lambda t: None if t is None else t.cuda()
    kw = dict(cu_seqlens=c(p["cu"]), initial_state=c(p["h0"]), input_scale=p["mode"])
    x, z = c(p["x"]), c(p["decay"])
    res = []
    for fn in fns:
        fin = torch.full_like(kw["initial_state"], 7.0)
        res.append((fn(x, z, final_state=fin, **kw), fin))
    _, chunks = g.gdn_scan(x, z, want_chunk_states=True, **kw)
    return res, g.gdn_scan_backward(c(d_out), x, z, chunks, **kw)


def near(got, want):
    tol = TOL + ref.ROUND[got.dtype]
    got = got.double().cpu().reshape(want.shape)
    assert bool(torch.isfinite(got).all())
    return bool(((got - want).abs() <= tol * want.abs() + 2.0 ** -126).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 70, 4096])
@pytest.mark.parametrize("name", [k for k in patterns() if k != "far beyond"])
def test_small_states_grow(name, D, dt):
    import gated_delta_rule_gate_gb300 as g
    gen = torch.Generator().manual_seed(D)
    rand = lambda *s: (0.5 + torch.rand(*s, generator=gen)) * 1e-25
    typed = lambda t: t.to(ref.DT[dt])
    one = patterns()[name]
    # a request of its own before and after, which begin and end inside a tile
    T = len(one)
    z = torch.cat([torch.full((21,), -0.3), one, torch.full((50,), -0.3)])[:, None].repeat(1, D)
    z = z * (1 + 0.01 * torch.rand(1, D, generator=gen))
    p = {"x": typed(rand(T + 71, D)), "decay": typed(z), "beta": None, "bias": None, "scale": None, "mode": "none",
         "sigmoid": False, "spans": [(0, 21), (21, 21 + T), (21 + T, T + 71)], "rows": [0, 1, 2], "nrows": 3,
         "h0": rand(3, D), "cu": torch.tensor([0, 21, 21 + T, T + 71], dtype=torch.int32)}
    d_out = typed(rand(T + 71, D))
    want, fin, grads = ref.scan(p, (d_out, None))
    assert float(want.max()) < 1e38 and float(grads["dx"].max()) < 1e38  # numbers that fp32 has
    res, got = run(p, d_out, (g.gdn_scan, g.gdn_scan_step))
    for out, end in res:
        assert near(out, want) and near(end, fin)
    assert near(got.dx, grads["dx"]) and near(got.d_initial_state, grads["d_initial_state"])
    assert near(got.d_decay, grads["d_decay"])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 70, 4096])
@pytest.mark.parametrize("name", list(patterns()))
def test_zeros_stay_zeros(name, D, dt):
    """No input and no state: zeros, whatever they are multiplied by; so are the gradients."""
    import gated_delta_rule_gate_gb300 as g
    z = patterns()[name][:, None].repeat(1, D).to(ref.DT[dt])
    zero = torch.zeros_like(z)
    p = {"x": zero, "decay": z, "mode": "none", "h0": torch.zeros(1, D), "cu": None}
    res, got = run(p, zero, (g.gdn_scan, g.gdn_scan_step))
    for out, end in res:
        assert torch.equal(out.cpu(), zero) and not bool(end.any())
    assert not bool(got.dx.any()) and not bool(got.d_decay.any()) and not bool(got.d_initial_state.any())
    # the last token's input stands alone
    p["x"] = zero.clone()
    p["x"][-1] = 3.0
    res, _ = run(p, zero, (g.gdn_scan, g.gdn_scan_step))
    for out, end in res:
        assert torch.equal(out.cpu(), p["x"]) and bool((end == 3.0).all())
