"""gdn_scan, gdn_scan_step and gdn_scan_backward value for value, each against a bound of its own
that is carried along the 64-bit token loop: an error in a channel of small values, or one far
above what fp32 leaves, is seen.

The bounds, in U = 2^-24 relative to the factor or term they stand at:
  softplus(z), |z| the size of decay + bias: the sum's rounding |z|, e^-|z| (4 + 1.25 |z|), the
      polynomial 3, and a rounding or two: 12 + 4 |z|;  g = scale softplus 1 more (0 without)
  a = e^g: 4 + 1.25 |g|, |g| times g's own, and 4 for the products it goes through
  e^g - 1: 10 and g's own where |g| <= 1/5; beyond, also a's rounding over what is left of 1
  n: that of e^g - 1, and 8 for the square root;  sigmoid(y): 8 + 1.25 |y|
  a run's factor is good to 2 (4 + 1.25 |G|) with G the sum of its g, less than its tokens' together.
The state's bound is b_t = a b_{t-1} + (a's) |a h_{t-1}| + (u's) |u|, the gradient's the same from the
right.  All bounds are doubled, for products of errors; 16-bit results add their rounding."""
import math

import pytest
import torch

import layer_reference as ref
import test_scan as fwd
import test_scan_backward as bwd

U = 2.0 ** -24


def factors(p, z, beta):
    """Relative bounds (in U) of a, n, i, the derivative n', sigmoid(z) scale, softplus."""
    zero = torch.zeros_like(z)
    raw = p["bias"] is not None
    if raw:
        s = z + p["bias"].double()
        soft = torch.logaddexp(s, zero)
        g = p["scale"].double() * soft
        c_soft = 12 + 4 * s.abs()
        c_g = c_soft + 1
        left = torch.exp(-soft) / -torch.expm1(-soft)
        c_slope = 12 + c_soft + torch.where(soft > 0.19, (5 + 1.25 * soft) * left, zero)
    else:
        g, c_g, c_soft, c_slope = z, zero, zero, zero
    a = torch.exp(g)
    c_a = 8 + 1.25 * g.abs() + g.abs() * c_g
    m = torch.expm1(g).abs()
    c_m = 10 + c_g + torch.where(g.abs() > 0.19, (5 + 1.25 * g.abs() + g.abs() * c_g) * a / m, zero)
    c_n = {"none": zero, "lerp": c_m, "unit": c_m + 8}[p["mode"]]
    c_dn = {"none": zero, "lerp": c_a, "unit": 2 * c_a + c_n + 4}[p["mode"]]
    c_i = zero if beta is None or not p["sigmoid"] else 8 + 1.25 * beta.abs()
    return c_a, c_n, c_i, c_dn, c_slope, c_soft


def carried(p, d_out, d_fin):
    """{name: (value, bound)} of every result, 64 bits."""
    D = p["x"].shape[-1]
    x, z, beta = (ref.flat(p[k], D) for k in ("x", "decay", "beta"))
    T = x.shape[0]
    dout, dfin = ref.flat(d_out, D), ref.flat(d_fin, D)
    new = lambda: torch.full((T, D), math.nan, dtype=torch.double)
    val = {k: new() for k in ("out", "dx", "d_decay", "d_beta")}
    err = {k: new() for k in val}
    for k in ("fin", "d_initial_state"):
        val[k], err[k] = (torch.full((p["nrows"], D), math.nan, dtype=torch.double) for _ in range(2))
    for k in ("d_gate_bias", "d_gate_scale"):
        val[k], err[k] = torch.zeros(D, dtype=torch.double), torch.zeros(D, dtype=torch.double)
    for (t0, t1), row in zip(p["spans"], p["rows"]):
        h, b = p["h0"][row].double(), torch.zeros(D, dtype=torch.double)
        prev = []
        for t in range(t0, t1):
            y = None if beta is None else beta[t]
            a, n, _, i, _, _, _ = ref.gate_terms(p, z[t], y)
            c_a, c_n, c_i, _, _, _ = factors(p, z[t], y)
            prev.append((h, b))
            u = n * i * x[t]
            h, b = a * h + u, a * b + U * (c_a * (a * h).abs() + (c_n + c_i + 4) * u.abs())
            val["out"][t], err["out"][t] = h, b
        val["fin"][row], err["fin"][row] = h, b
        c, b = dfin[row], torch.zeros(D, dtype=torch.double)
        for t in reversed(range(t0, t1)):
            y = None if beta is None else beta[t]
            a, n, dn, i, di, soft, dgdz = ref.gate_terms(p, z[t], y)
            c_a, c_n, c_i, c_dn, c_slope, c_soft = factors(p, z[t], y)
            hp, hb = prev[t - t0]
            dh, e = dout[t] + c, b + U * (dout[t] + c).abs()
            dx = n * i * dh
            val["dx"][t], err["dx"][t] = dx, (n * i).abs() * e + U * (c_n + c_i + 3) * dx.abs()
            one, two = a * hp * dh, dn * i * x[t] * dh
            e_dg = (a * hp).abs() * e + (a * dh).abs() * hb + U * (c_a + 3) * one.abs() \
                + (dn * i * x[t]).abs() * e + U * (c_dn + c_i + 4) * two.abs()
            dg = one + two
            dz, e_dz = dg * dgdz, e_dg * dgdz.abs() + U * (c_slope + 4) * (dg * dgdz).abs()
            val["d_decay"][t], err["d_decay"][t] = dz, e_dz
            if di is not None:
                db = n * x[t] * dh * di
                # i (1 - i), formed as i - i i
                c_di = 0 if not p["sigmoid"] else (c_i * (1 + i) + 2) / (1 - i)
                val["d_beta"][t] = db
                err["d_beta"][t] = (n * x[t] * di).abs() * e + U * (c_n + c_di + 4) * db.abs()
            if soft is not None:
                val["d_gate_bias"] += dz
                err["d_gate_bias"] += e_dz + U * T * dz.abs()  # a sum of T terms
                val["d_gate_scale"] += dg * soft
                err["d_gate_scale"] += soft * e_dg + U * (c_soft + T) * (dg * soft).abs()
            c, b = a * dh, a * e + U * c_a * (a * dh).abs()
        val["d_initial_state"][row], err["d_initial_state"][row] = c, b
    return val, err


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("mode", ["none", "lerp", "unit"])
@pytest.mark.parametrize("raw", [True, False])
@pytest.mark.parametrize("beta", [None, "plain", "sigmoid"])
def test_within_the_carried_bounds(act, mode, raw, beta):
    import gated_delta_rule_gate_gb300 as g
    p = fwd.draw(900, 72, lengths=[230, 1, 140], act=act, mode=mode, raw=raw, beta=beta, gate="same")
    # channels of small values beside large ones
    size = torch.logspace(-6, 2, 72)
    p["h0"] = p["h0"] * size
    if act != "f16":
        p["x"] = (p["x"].float() * size).to(p["x"].dtype)
    d_out, d_fin, got = bwd.run(p, 5)
    val, err = carried(p, d_out, d_fin)
    results = {"dx": got.dx, "d_decay": got.d_decay, "d_beta": got.d_beta, "d_gate_bias": got.d_gate_bias,
               "d_gate_scale": got.d_gate_scale, "d_initial_state": got.d_initial_state}
    for fn in (g.gdn_scan, g.gdn_scan_step):
        results["out"], results["fin"] = fwd.call(p, fn)
        for name, t in results.items():
            if t is None:
                continue
            least = 2.0 ** -24 if t.dtype == torch.float16 else 2.0 ** -126  # of its smallest numbers
            room = ref.ROUND[t.dtype] * val[name].abs() + least
            off = (t.detach().cpu().double().reshape(val[name].shape) - val[name]).abs()
            assert bool((off <= 2 * err[name] + room).all()), (name, float((off / (2 * err[name] + room)).max()))
