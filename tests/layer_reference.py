"""Plain 64-bit forms of the recurrent-layer operators (torch on the CPU, token
by token, written from the formulas), and helpers to draw their inputs."""
import math

import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# one rounding on store, relative to the value
ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def tokens_of(lengths=None, cu=None, T=None, S=None, seq_lens=None):
    """[(begin, end)] of each request."""
    if S is not None:
        return [(b * S, b * S + n) for b, n in enumerate(seq_lens)]
    if cu is None:
        cu = [0]
        for n in lengths:
            cu.append(cu[-1] + n)
    c = [min(max(v, 0), T) for v in cu]
    return [(a, max(a, b)) for a, b in zip(c, c[1:])]


def gate_terms(p, z, beta):
    """a, n, dn/dg, i, di/dbeta, softplus, dg/dz of gate inputs z, beta (64 bits)."""
    one = torch.ones_like(z)
    soft = slope = None
    g, dgdz = z, one
    if p["bias"] is not None:
        s = z + p["bias"].double()
        soft = torch.logaddexp(s, torch.zeros_like(s))
        slope = torch.sigmoid(s)
        g, dgdz = p["scale"].double() * soft, p["scale"].double() * slope
    a = torch.exp(g)
    if p["mode"] == "lerp":
        n, dn = -torch.expm1(g), -a
    elif p["mode"] == "unit":
        q = torch.clamp(-torch.expm1(2 * g), min=0)
        n = torch.sqrt(q)
        dn = torch.where(q > 0, -a * a / torch.where(q > 0, n, one), torch.zeros_like(n))
    else:
        n, dn = one, torch.zeros_like(a)
    i, di = one, None
    if beta is not None:
        i, di = beta, one
        if p["sigmoid"]:
            i = torch.sigmoid(beta)
            di = i * (1 - i)
    return a, n, dn, i, di, soft, dgdz


def flat(t, D):
    return None if t is None else t.detach().cpu().double().reshape(-1, D)


def scan(p, grad=None):
    """p: x, decay, beta, bias, scale, mode, sigmoid, spans, rows (of each request, None: skipped), h0, nrows.
    Returns out (NaN where no request is), final rows (NaN where untouched); with ``grad`` = (d_out,
    d_final or None) also a dict of the gradients."""
    D = p["x"].shape[-1]
    x, z, beta = flat(p["x"], D), flat(p["decay"], D), flat(p["beta"], D)
    T = x.shape[0]
    out = torch.full((T, D), math.nan, dtype=torch.double)
    fin = torch.full((p["nrows"], D), math.nan, dtype=torch.double)
    g = None
    if grad is not None:
        dout, dfin = flat(grad[0], D), flat(grad[1], D)
        g = {k: torch.full((T, D), math.nan, dtype=torch.double) for k in ("dx", "d_decay", "d_beta")}
        g["d_gate_bias"] = torch.zeros(D, dtype=torch.double)
        g["d_gate_scale"] = torch.zeros(D, dtype=torch.double)
        g["sum_of_sizes"] = torch.zeros(2, D, dtype=torch.double)  # of the terms of the two sums
        g["d_initial_state"] = torch.full((p["nrows"], D), math.nan, dtype=torch.double)
    for (t0, t1), row in zip(p["spans"], p["rows"]):
        if row is None:
            continue
        h = p["h0"][row].detach().cpu().double().clone() if p["h0"] is not None else torch.zeros(D, dtype=torch.double)
        prev = []
        for t in range(t0, t1):
            a, n, _, i, _, _, _ = gate_terms(p, z[t], None if beta is None else beta[t])
            prev.append(h)
            h = a * h + n * i * x[t]
            out[t] = h
        fin[row] = h
        if g is None:
            continue
        c = dfin[row].clone() if dfin is not None else torch.zeros(D, dtype=torch.double)
        for t in reversed(range(t0, t1)):
            a, n, dn, i, di, soft, dgdz = gate_terms(p, z[t], None if beta is None else beta[t])
            dh = dout[t] + c
            dg = a * prev[t - t0] * dh + dn * i * x[t] * dh
            g["dx"][t] = n * i * dh
            g["d_decay"][t] = dg * dgdz
            if di is not None:
                g["d_beta"][t] = n * x[t] * dh * di
            if soft is not None:
                g["d_gate_scale"] += dg * soft
                g["d_gate_bias"] += dg * dgdz
                g["sum_of_sizes"] += torch.stack([(dg * dgdz).abs(), (dg * soft).abs()])
            c = a * dh
        g["d_initial_state"][row] = c
    return (out, fin) if g is None else (out, fin, g)


def rel(x, ref):
    """max |x - ref| / max |ref| where ref is a number; inf if x is not one there."""
    x = x.detach().cpu().double().reshape(ref.shape)
    at = ~torch.isnan(ref)
    if not bool(at.any()):
        return 0.0
    if not bool(torch.isfinite(x[at]).all()):
        return math.inf
    top = float(ref[at].abs().max())
    return float((x[at] - ref[at]).abs().max()) / (top if top > 0 else 1.0)
