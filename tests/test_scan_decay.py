"""The decay keeps its digits where it is small: value for value, relative to each value,
on states that no input adds to.

Tolerances.  A token's a = e^g goes through g log2(e), rounded to 2^-24 of itself with a
constant that is 0.22 2^-24 off, and a power of two that is good to 2^-22: (4 + 1.25 |g|) 2^-24
of a.  In the raw arm g = scale softplus(z) carries the same of e^-|z| (|z| <= 4: 9), the
polynomial's 3, the sum's rounding (4) and a product's 1, 2^-24 each, of itself: 18 |g| 2^-24
more.  Each token multiplies once or twice more.  What all terms of one sign make of that adds
over the tokens that a value has gone through, all of them at most."""
import pytest
import torch

import layer_reference as ref

U = 2.0 ** -24


def draw(T, D, raw, lo, hi, seed):
    """Decays of all channels between lo and hi a token, positive states."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=gen)
    p = {"x": torch.zeros(T, D), "beta": None, "bias": None, "scale": None, "mode": "none", "sigmoid": False,
         "spans": [(0, T)], "rows": [0], "nrows": 1, "h0": 0.5 + rand(1, D)}
    if raw:
        p["decay"], p["bias"] = 3 * rand(T, D) - 1, 2 * rand(D) - 1
        p["scale"] = (lo + (hi - lo) * rand(D)) / 4
        g = p["scale"].double() * torch.logaddexp((p["decay"] + p["bias"]).double(), torch.zeros(1, dtype=torch.double))
    else:
        p["decay"] = lo + (hi - lo) * rand(T, D)
        g = p["decay"].double()
    error = 4 + 1.25 * g.abs() + (18 * g.abs() if raw else 0) + 4
    return p, U * (error.sum(0) + 8)


CASES = [(1, -5, -30), (2, -8, -30), (3, -0.1, -25), (17, -1, -4), (40, -0.2, -1.5), (130, -0.01, -0.6),
         (1, -30, -80)]


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["none", "lerp", "unit"])
@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("T,lo,hi", CASES)
@pytest.mark.parametrize("D", [64, 131])
def test_states_and_gradients_value_for_value(T, lo, hi, raw, mode, D):
    import gated_delta_rule_gate_gb300 as g
    p, tol = draw(T, D, raw, lo, hi, 7 * T + D)
    p["mode"] = mode
    d_out = 0.5 + torch.rand(T, D, generator=torch.Generator().manual_seed(T))
    want, fin, grads = ref.scan(p, (d_out, None))
    c = lambda t: None if t is None else t.cuda()
    kw = dict(gate_bias=c(p["bias"]), gate_scale=c(p["scale"]), input_scale=mode, initial_state=c(p["h0"]))
    x, z = c(p["x"]), c(p["decay"])

    def near(got, want):
        return bool(((got.double().cpu() - want).abs() <= tol * want.abs() + 2.0 ** -126).all())

    end = torch.zeros(1, D, device="cuda")
    for fn in (g.gdn_scan_step, g.gdn_scan):
        out = fn(x, z, final_state=end.zero_(), **kw)
        assert near(out, want) and near(end, fin)
    _, chunks = g.gdn_scan(x, z, want_chunk_states=True, **kw)
    got = g.gdn_scan_backward(c(d_out), x, z, chunks, **kw)
    assert near(got.d_initial_state, grads["d_initial_state"])
    assert near(got.d_decay, grads["d_decay"])
