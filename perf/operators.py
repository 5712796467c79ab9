"""Cases of the recurrent-layer operators: what a pass reads and returns, its plain form, and its 64-bit value.

Five operators around a gated linear recurrence of vector state, as a layer is served and trained:

  step   gdn_scan_step      one or a few tokens per request, state rows of a slab updated in place (serving)
  scan   gdn_scan           whole sequences (prefill)
  train  gdn_scan + gdn_scan_backward       a training pass through the recurrence
  norm   gdn_rmsnorm        residual addition, root-mean-square norm, output in 8 bits with scales (serving)
  normtrain  gdn_rmsnorm + gdn_rmsnorm_backward   a training pass through the norm
  clip   gdn_grad_clip      the global gradient norm over many tensors, and clipping

Per channel: g = decay, or gate_scale * softplus(decay + gate_bias); a = exp(g); n = 1, 1 - a ("lerp") or
sqrt(1 - a^2) ("unit"); i = 1 or sigmoid(beta); h_t = a_t h_{t-1} + n_t i_t x_t.

`own` False: elementary torch operations in 32 bits, rounded once at the end.  True: the calls of the package.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SZ = {"f32": 4, "f16": 2, "bf16": 2}
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # rows (groups) of zeros get a positive scale
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest serving call: one request, one token, the layer width of 16 heads of 128
        {"name": "step-1", "op": "step", "requests": 1, "tokens": 1, "channels": 2048, "slots": 8, "dtype": "f16",
         "gate_dtype": "f16", "input_gate": True, "input_scale": "unit"},
        # the decode batch: 256 requests of one token in a slab of 1024 rows, 32 heads of 128
        {"name": "step-256", "op": "step", "requests": 256, "tokens": 1, "channels": 4096, "slots": 1024,
         "dtype": "f16", "gate_dtype": "f16", "input_gate": True, "input_scale": "unit"},
        # a small ragged prefill of odd sizes in 32 bits, some requests empty, log decay given
        {"name": "scan-odd", "op": "scan", "requests": 7, "tokens": 1001, "channels": 517, "dtype": "f32",
         "gate_dtype": "f32", "gate": "log", "input_gate": False, "input_scale": "none", "layout": "packed",
         "states": True},
        # the ragged prefill: 8 requests of 16384 tokens together, 32 heads of 128
        {"name": "scan-ragged", "op": "scan", "requests": 8, "tokens": 16384, "channels": 4096, "dtype": "f16",
         "gate_dtype": "f16", "gate": "raw", "input_gate": True, "input_scale": "unit", "layout": "packed",
         "states": True},
        # a training pass over odd sizes in 32 bits with padded rows
        {"name": "train-odd", "op": "train", "requests": 3, "tokens": 999, "channels": 1000, "dtype": "f32",
         "gate_dtype": "f32", "gate": "raw", "input_gate": True, "input_scale": "lerp", "layout": "padded",
         "states": True},
        # a training pass over four sequences of 8192 tokens, 16 heads of 128
        {"name": "train-long", "op": "train", "requests": 4, "tokens": 32768, "channels": 2048, "dtype": "bf16",
         "gate_dtype": "bf16", "gate": "raw", "input_gate": True, "input_scale": "unit", "layout": "uniform",
         "states": False},
        # the decode batch's norm: 256 rows, an 8-bit output with one scale a row
        {"name": "norm-256", "op": "norm", "rows": 256, "dim": 4096, "dtype": "f16", "residual": "f16", "group": 0},
        # the long prefill's norm: a 32-bit residual stream, an 8-bit output with a scale for each 128 columns
        {"name": "norm-long", "op": "norm", "rows": 32768, "dim": 2048, "dtype": "bf16", "residual": "f32",
         "group": 128},
        # a training pass through the norm at odd sizes, 32 bits
        {"name": "normtrain-odd", "op": "normtrain", "rows": 1001, "dim": 1531, "dtype": "f32", "residual": "f32"},
        # a training pass through the norm over four sequences of 8192 tokens
        {"name": "normtrain-long", "op": "normtrain", "rows": 32768, "dim": 2048, "dtype": "bf16",
         "residual": "bf16"},
        # the gradients of one small layer, 32 bits, odd sizes, under the bound (nothing to clip)
        {"name": "clip-layer", "op": "clip", "layers": 1, "width": 517, "dtype": "f32", "clips": False},
        # the gradients of 24 layers of width 2048 in 16 bits, clipped
        {"name": "clip-model", "op": "clip", "layers": 24, "width": 2048, "dtype": "bf16", "clips": True},
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n == 3072 else n


def _width(rng, lo, hi):
    """A channel count: a multiple of 128 half the time, any number otherwise."""
    d = _log(rng, lo, hi)
    even = max(128, d // 128 * 128)
    return even if rng.random() < 0.5 and even != 3072 else d


def draw(rng):
    op = rng.choice(["step", "scan", "train", "norm", "normtrain", "clip"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    gate_dtype = dtype if rng.random() < 0.7 else "f32"
    if op == "step":
        requests = _log(rng, 1, 512)
        return {"op": op, "requests": requests, "tokens": rng.choice([1, 1, 1, 2, 4]),
                "channels": _width(rng, 200, 5000), "slots": requests * rng.choice([1, 2, 4]), "dtype": dtype,
                "gate_dtype": gate_dtype, "input_gate": rng.random() < 0.7,
                "input_scale": rng.choice(["none", "lerp", "unit"])}
    if op in ("scan", "train"):
        channels = _width(rng, 200, 5000)
        tokens = min(_log(rng, 200, 32768), (1 << 26) // channels)
        requests = min(_log(rng, 1, 32), tokens)
        layout = rng.choice(["packed", "packed", "padded", "uniform"])
        if layout != "packed":
            tokens -= tokens % requests
        return {"op": op, "requests": requests, "tokens": tokens, "channels": channels, "dtype": dtype,
                "gate_dtype": gate_dtype, "gate": rng.choice(["log", "raw"]), "input_gate": rng.random() < 0.6,
                "input_scale": rng.choice(["none", "lerp", "unit"]), "layout": layout,
                "states": rng.random() < 0.6}
    if op == "clip":
        width = _log(rng, 100, 2048)
        return {"op": op, "layers": _log(rng, 1, max(1, min(48, 24 * 2048 ** 2 // (2 * width ** 2)))),
                "width": width, "dtype": dtype, "clips": rng.random() < 0.7}
    dim = _width(rng, 200, 8192)
    rows = min(_log(rng, 1 if op == "norm" else 64, 32768), (1 << 25) // dim)
    case = {"op": op, "rows": rows, "dim": dim, "dtype": dtype,
            "residual": rng.choice([dtype, "f32"]) if op == "normtrain" else rng.choice([dtype, "f32", "none"])}
    if op == "norm":
        case["group"] = rng.choice([0, 128])
    return case


# ------------------------------------------------------------------ inputs
def _lengths(case, rng):
    """Request lengths: even rows, or drawn and rescaled to sum to the tokens, one in five requests empty."""
    B, T = case["requests"], case["tokens"]
    if case["layout"] == "uniform":
        return [T // B] * B
    if case["layout"] == "padded":
        S = T // B
        return [S if b == 0 else rng.randint(0, S) for b in range(B)]
    raw = [0.0 if B > 4 and rng.random() < 0.2 else rng.uniform(0.02, 1.0) for _ in range(B)]
    raw[rng.randrange(B)] = 1.0
    n = [int(r * T / sum(raw)) for r in raw]
    n[max(range(B), key=lambda b: n[b])] += T - sum(n)
    return n


def _shapes(case):
    """The gradient tensors of a stack of recurrent blocks: projections, gate parameters, norm weights."""
    w = case["width"]
    block = [(w, w), (w, w), (w, w), (w, w), (w,), (w,), (w,)]
    return block * case["layers"]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rng = random.Random(int(seed))
    dt = DT[case["dtype"]]

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    def uniform(*shape, lo, hi):
        return lo + (hi - lo) * torch.rand(*shape, generator=gen, device=dev)

    op = case["op"]
    if op == "clip":
        grads = [normal(*s, std=0.02) for s in _shapes(case)]
        # a fixed bound, far under or far over the norm that such gradients have
        total = sum(g.numel() for g in grads)
        bound = 0.02 * math.sqrt(total) * (0.1 if case["clips"] else 10.0)
        return {"case": case, "grads": grads, "max_norm": bound, "out": [torch.zeros_like(g) for g in grads],
                "norm": torch.zeros(1, device=dev)}
    if op in ("norm", "normtrain"):
        N, D = case["rows"], case["dim"]
        s = {"case": case, "x": normal(N, D), "weight": normal(D, std=0.1) + 1}
        s["residual"] = None if case["residual"] == "none" else normal(N, D, dtype=DT[case["residual"]], std=2.0)
        if op == "normtrain":
            s["dy"] = normal(N, D)
            s["dres"] = normal(N, D, dtype=DT[case["residual"]])
        return s

    B, D = case["requests"], case["channels"]
    gd = DT[case["gate_dtype"]]
    if op == "step":
        L = case["tokens"]
        T = B * L
        lengths = [L] * B
        case = dict(case, gate="raw", layout="packed", states=True)
        rows = case["slots"]
        order = list(range(rows))
        rng.shuffle(order)
        slots = torch.tensor(order[:B], dtype=torch.int32, device=dev)
    else:
        T, rows, slots = case["tokens"], B, None
        lengths = _lengths(case, rng)
    lead = (T,) if case["layout"] == "packed" else (B, T // B)
    s = {"case": case, "x": normal(*lead, D), "slots": slots, "lengths": lengths, "cu": None, "seq_lens": None}
    if case["layout"] == "packed":
        cu = [0]
        for n in lengths:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    elif case["layout"] == "padded":
        s["seq_lens"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    if case["gate"] == "raw":
        # memories from a few tokens to hundreds, as trained gates have
        s["decay"] = normal(*lead, D, dtype=gd)
        s["bias"] = uniform(D, lo=-2.0, hi=2.0)
        s["scale"] = -torch.exp(uniform(D, lo=-4.0, hi=2.0))
    else:
        s["decay"] = (-torch.exp(uniform(*lead, D, lo=-7.0, hi=1.0))).to(gd)
        s["bias"] = s["scale"] = None
    s["beta"] = normal(*lead, D, dtype=gd) if case["input_gate"] else None
    s["h0"] = normal(rows, D, dtype=torch.float32) if case["states"] else None
    s["hT"] = s["h0"] if op == "step" else torch.zeros(rows, D, device=dev) if case["states"] else None
    s["out"] = torch.zeros_like(s["x"])
    # which request each token belongs to and where that request's tokens begin and end, for the plain form
    S = lead[1] if len(lead) == 2 else 0
    begin = [sum(lengths[:b]) if not S else b * S for b in range(B)]
    s["begin"], s["end"] = begin, [p + n for p, n in zip(begin, lengths)]
    first = torch.tensor([p for p, n in zip(begin, lengths) if n], dtype=torch.int64, device=dev)
    last = torch.tensor([p + n - 1 for p, n in zip(begin, lengths) if n], dtype=torch.int64, device=dev)
    owner = torch.tensor([b for b, n in enumerate(lengths) if n], dtype=torch.int64, device=dev)
    s["first"], s["last"] = first, last
    s["row"] = slots.long()[owner] if slots is not None else owner
    covered = torch.zeros(T, 1, dtype=torch.bool, device=dev)
    for p, n in zip(begin, lengths):
        covered[p:p + n] = True
    s["covered"] = covered
    if op == "train":
        s["dout"] = normal(*lead, D)
        s["dhT"] = normal(rows, D, dtype=torch.float32) if case["states"] else None
        for k in ("dx", "ddecay", "dbeta"):
            src = {"dx": "x", "ddecay": "decay", "dbeta": "beta"}[k]
            s[k] = torch.zeros_like(s[src]) if s[src] is not None else None
    return s


# ------------------------------------------------------------------ plain forms, 32 bits
def _doubling(A, H, reach):
    """H_t <- sum over s <= t of (A_t ... A_{s+1}) H_s along the first axis, by doubling the distance that is
    covered up to the longest request."""
    d = 1
    while d < reach:
        H = torch.cat([H[:d], H[d:] + A[d:] * H[:-d]])
        A = torch.cat([A[:d], A[d:] * A[:-d]])
        d *= 2
    return H


def _gates(s, real=torch.float32):
    """g, softplus, its derivative, a, n, dn/dg and i of every token and channel, [T, D]."""
    D = s["x"].shape[-1]
    z = s["decay"].reshape(-1, D).to(real)
    if s["bias"] is not None:
        z = z + s["bias"].to(real)
        soft = torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))
        slope = torch.where(z >= 0, 1 / (1 + torch.exp(-z.abs())), 1 - 1 / (1 + torch.exp(-z.abs())))
        g = s["scale"].to(real) * soft
    else:
        g, soft, slope = z, None, None
    a = torch.exp(g)
    mode = s["case"]["input_scale"]
    if mode == "none":
        n = dn = None
    elif mode == "lerp":
        n, dn = -torch.expm1(g), -a
    else:
        n = torch.sqrt(-torch.expm1(2 * g))
        dn = torch.where(n > 0, -a * a / torch.where(n > 0, n, torch.ones_like(n)), torch.zeros_like(n))
    i = None if s["beta"] is None else 1 / (1 + torch.exp(-s["beta"].reshape(-1, D).to(real)))
    return g, soft, slope, a, n, dn, i


def _plain_scan(s):
    """Every token's state and the state before it (fp32 [T, D]), and what the gradient reuses."""
    D = s["x"].shape[-1]
    x = s["x"].reshape(-1, D).float()
    gates = _gates(s)
    a, n, i = gates[3], gates[4], gates[6]
    u = x if i is None else i * x
    u = u if n is None else n * u
    cov, first = s["covered"], s["first"]
    zero = torch.zeros((), device=x.device)
    u = torch.where(cov, u, zero)
    A = torch.where(cov, a, zero)
    start = torch.zeros(len(first), D, device=x.device) if s["h0"] is None else s["h0"][s["row"]]
    u[first] += a[first] * start
    A[first] = 0
    h = _doubling(A, u, max(s["lengths"]))
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    prev[first] = start
    return x, gates, h, prev


def _plain_final(s, h):
    if s["hT"] is None:
        return None
    fin = s["h0"].clone() if s["h0"] is not s["hT"] else s["hT"]
    fin[s["row"]] = h[s["last"]]
    return fin


def _plain_train(s):
    D = s["x"].shape[-1]
    x, (g, soft, slope, a, n, dn, i), h, prev = _plain_scan(s)
    cov, first, last = s["covered"], s["first"], s["last"]
    zero = torch.zeros((), device=x.device)
    do = torch.where(cov, s["dout"].reshape(-1, D).float(), zero)
    if s["dhT"] is not None:
        do[last] += s["dhT"][s["row"]]
    # dh_t = do_t + a_{t+1} dh_{t+1}: the same sums over the reversed axis, the factors one token on
    nxt = torch.where(cov, a, zero)
    nxt[first] = 0
    nxt = torch.cat([nxt[1:], torch.zeros_like(nxt[:1])])
    dh = _doubling(nxt.flip(0), do.flip(0), max(s["lengths"])).flip(0)
    dg = a * prev * dh
    w = torch.ones_like(x) if n is None else n
    inner = x if i is None else i * x
    if dn is not None:
        dg = dg + dn * inner * dh
    out = {"dx": w * dh if i is None else w * i * dh}
    if i is not None:
        out["dbeta"] = w * x * dh * i * (1 - i)
    if s["bias"] is not None:
        dz = dg * s["scale"] * slope
        out["ddecay"] = dz
        out["dbias"] = torch.where(cov, dz, zero).sum(0)
        out["dscale"] = torch.where(cov, dg * soft, zero).sum(0)
    else:
        out["ddecay"] = dg
    for k in ("dx", "ddecay", "dbeta"):
        if k in out:
            out[k] = torch.where(cov, out[k], zero).to(s[k].dtype).view_as(s[k])
    if s["h0"] is not None:
        dh0 = torch.zeros_like(s["h0"]) if s["dhT"] is None else s["dhT"].clone()
        dh0[s["row"]] = a[first] * dh[first]
        out["dh0"] = dh0
    out["out"] = torch.where(cov, h, zero).to(s["x"].dtype).view_as(s["x"])
    out["hT"] = _plain_final(s, h)
    return out


def _quantised(y, group):
    """y in e4m3 and the scales: per row (group 0), or per `group` columns (the last group may be short)."""
    N, D = y.shape
    if not group:
        scale = torch.clamp(y.abs().amax(1), min=AMAX_FLOOR) / E4M3_MAX
        return (y / scale[:, None]).to(torch.float8_e4m3fn), scale
    pad = -D % group
    z = torch.nn.functional.pad(y, (0, pad)).view(N, -1, group)
    scale = torch.clamp(z.abs().amax(2), min=AMAX_FLOOR) / E4M3_MAX
    return (z / scale[:, :, None]).view(N, -1)[:, :D].contiguous().to(torch.float8_e4m3fn), scale


def _plain_norm(s):
    r = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    rstd = torch.rsqrt(r.square().mean(1, keepdim=True) + EPS)
    return r, rstd, r * rstd * s["weight"].float()


def _plain(s):
    op = s["case"]["op"]
    if op in ("step", "scan"):
        _, _, h, _ = _plain_scan(s)
        out = torch.where(s["covered"], h, torch.zeros((), device=h.device)).to(s["x"].dtype).view_as(s["x"])
        return {"out": out, "hT": _plain_final(s, h)}
    if op == "train":
        return _plain_train(s)
    if op == "norm":
        r, _, y = _plain_norm(s)
        q, scale = _quantised(y, s["case"]["group"])
        return {"out": q, "scales": scale, "residual": None if s["residual"] is None else r.to(s["residual"].dtype)}
    if op == "normtrain":
        r, rstd, y = _plain_norm(s)
        res = r.to(s["residual"].dtype)
        xhat = res.float() * rstd
        wdy = s["weight"].float() * s["dy"].float()
        dr = rstd * (wdy - xhat * (wdy * xhat).mean(1, keepdim=True)) + s["dres"].float()
        dw = (s["dy"].float() * xhat).sum(0)
        return {"out": y.to(s["x"].dtype), "residual": res, "dr": dr.to(res.dtype), "dweight": dw}
    norm = torch.sqrt(sum(g.float().square().sum() for g in s["grads"]))
    coef = torch.clamp(s["max_norm"] / (norm + EPS), max=1.0)
    return {"norm": norm.view(1), "out": _first_and_last([(g.float() * coef).to(g.dtype) for g in s["grads"]])}


def _first_and_last(ts):
    """At most 60 of a long list of tensors: the first and the last 30."""
    return list(ts) if len(ts) <= 60 else list(ts[:30]) + list(ts[-30:])


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import gated_delta_rule_gate_gb300 as gdn
    case = s["case"]
    op = case["op"]
    if op == "clip":
        gdn.gdn_grad_clip(s["grads"], s["max_norm"], eps=EPS, out=s["out"], norm=s["norm"])
        return {"norm": s["norm"], "out": _first_and_last(s["out"])}
    if op == "norm":
        r = gdn.gdn_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS, out_dtype=torch.float8_e4m3fn,
                            group=case["group"])
        return {"out": r.out, "scales": r.scales, "residual": r.residual}
    if op == "normtrain":
        r = gdn.gdn_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS, want_rstd=True)
        b = gdn.gdn_rmsnorm_backward(s["dy"], r.residual, s["weight"], r.rstd, d_residual=s["dres"])
        return {"out": r.out, "residual": r.residual, "dr": b.dx, "dweight": b.dweight}
    gates = dict(beta=s["beta"], beta_sigmoid=s["beta"] is not None, gate_bias=s["bias"], gate_scale=s["scale"],
                 input_scale=case["input_scale"], cu_seqlens=s["cu"], initial_state=s["h0"])
    if op == "step":
        gdn.gdn_scan_step(s["x"], s["decay"], slot_ids=s["slots"], final_state=s["hT"], out=s["out"], **gates)
        return {"out": s["out"], "hT": s["hT"]}
    if op == "scan":
        gdn.gdn_scan(s["x"], s["decay"], seq_lens=s["seq_lens"], final_state=s["hT"], out=s["out"], **gates)
        return {"out": s["out"], "hT": s["hT"]}
    _, chunks = gdn.gdn_scan(s["x"], s["decay"], seq_lens=s["seq_lens"], final_state=s["hT"], out=s["out"],
                             want_chunk_states=True, **gates)
    b = gdn.gdn_scan_backward(s["dout"], s["x"], s["decay"], chunks, seq_lens=s["seq_lens"], d_final_state=s["dhT"],
                              dx=s["dx"], d_decay=s["ddecay"], d_beta=s["dbeta"], **gates)
    out = {"out": s["out"], "hT": s["hT"], "dx": b.dx, "ddecay": b.d_decay}
    if s["beta"] is not None:
        out["dbeta"] = b.d_beta
    if s["bias"] is not None:
        out["dbias"], out["dscale"] = b.d_gate_bias, b.d_gate_scale
    if s["h0"] is not None:
        out["dh0"] = b.d_initial_state
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def work(case):
    op, e = case["op"], SZ[case["dtype"]]
    if op == "clip":
        n = sum(math.prod(s) for s in _shapes(case))
        return {"bytes": 2 * e * n, "flops": 3 * n}
    if op in ("norm", "normtrain"):
        n = case["rows"] * case["dim"]
        r = 0 if case["residual"] == "none" else SZ[case["residual"]]
        if op == "norm":
            scales = case["rows"] * (1 if not case["group"] else -(-case["dim"] // case["group"]))
            return {"bytes": n * (e + 2 * r + 1) + 4 * scales + e * case["dim"], "flops": 7 * n}
        # x, residual in; out, residual out; dy, the gradient of the residual in; the gradient out (the
        # residual that the backward pass reads is the forward pass's output)
        return {"bytes": n * (e + r + e + r + e + r + r) + 8 * case["dim"], "flops": 16 * n}
    T = case["requests"] * case["tokens"] if op == "step" else case["tokens"]
    n, q = T * case["channels"], SZ[case["gate_dtype"]]
    gates = q * (2 if case["input_gate"] else 1)
    states = case["requests"] * case["channels"] * 4 * 2 if case.get("states", True) else 0
    if op == "train":
        # forward: x and the gates in, o out; backward: d_o in, the gradients of x and the gates out
        return {"bytes": n * (e + gates + e + e + e + gates) + 2 * states, "flops": 45 * n}
    return {"bytes": n * (2 * e + gates) + states, "flops": 15 * n}


# ------------------------------------------------------------------ 64 bits, token by token
def _exact_gates(s, t):
    """a, n, dn/dg, i, softplus and its slope of the tokens `t` (indices), 64 bits."""
    D = s["x"].shape[-1]
    z = s["decay"].reshape(-1, D)[t].double()
    soft = slope = None
    if s["bias"] is not None:
        z = z + s["bias"].double()
        soft, slope = torch.logaddexp(z, torch.zeros_like(z)), torch.sigmoid(z)
        z = s["scale"].double() * soft
    a, mode = torch.exp(z), s["case"]["input_scale"]
    one = torch.ones_like(a)
    if mode == "lerp":
        n, dn = -torch.expm1(z), -a
    elif mode == "unit":
        n = torch.sqrt(-torch.expm1(2 * z))
        dn = torch.where(n > 0, -a * a / torch.where(n > 0, n, one), torch.zeros_like(n))
    else:
        n, dn = one, torch.zeros_like(a)
    i = one if s["beta"] is None else torch.sigmoid(s["beta"].reshape(-1, D)[t].double())
    return a, n, dn, i, soft, slope


def _exact_recurrence(s):
    dev = s["x"].device
    D = s["x"].shape[-1]
    T = s["x"].numel() // D
    x = s["x"].reshape(-1, D)
    order = sorted((b for b in range(len(s["begin"])) if s["end"][b] > s["begin"][b]),
                   key=lambda b: s["begin"][b] - s["end"][b])
    slots = s["slots"].tolist() if s["slots"] is not None else list(range(len(s["begin"])))
    rows = torch.tensor([slots[b] for b in order], device=dev)
    starts = torch.tensor([s["begin"][b] for b in order], device=dev)
    lens = [s["end"][b] - s["begin"][b] for b in order]
    longest = lens[0] if lens else 0
    live = [sum(n > t for n in lens) for t in range(longest)]  # requests are ordered by length
    h = s["h0"].double()[rows] if s["h0"] is not None else torch.zeros(len(order), D, device=dev, dtype=torch.double)
    out = torch.zeros(T, D, device=dev, dtype=torch.double)
    train = s["case"]["op"] == "train"
    prev = torch.zeros_like(out) if train else None
    for t in range(longest):
        k = live[t]
        at = starts[:k] + t
        a, n, _, i, _, _ = _exact_gates(s, at)
        if train:
            prev[at] = h[:k]
        h[:k] = a * h[:k] + n * i * x[at].double()
        out[at] = h[:k]
    res = {"out": out.view(s["x"].shape), "hT": None}
    if s["hT"] is not None:
        res["hT"] = s["h0"].double().clone()
        res["hT"][rows] = h
    if not train:
        return res
    dout = s["dout"].reshape(-1, D)
    dx, dz = torch.zeros_like(out), torch.zeros_like(out)
    db = torch.zeros_like(out)
    dbias = torch.zeros(D, device=dev, dtype=torch.double)
    dscale = torch.zeros_like(dbias)
    c = s["dhT"].double()[rows] if s["dhT"] is not None else torch.zeros_like(h)
    for t in reversed(range(longest)):
        k = live[t]
        at = starts[:k] + t
        a, n, dn, i, soft, slope = _exact_gates(s, at)
        xt = x[at].double()
        dh = dout[at].double() + c[:k]
        dg = a * prev[at] * dh + dn * i * xt * dh
        dx[at] = n * i * dh
        db[at] = n * xt * dh * i * (1 - i)
        c[:k] = a * dh
        if soft is not None:
            dscale += (dg * soft).sum(0)
            dg = dg * s["scale"].double() * slope
            dbias += dg.sum(0)
        dz[at] = dg
    shape = s["x"].shape
    res |= {"dx": dx.view(shape), "ddecay": dz.view(shape)}
    if s["beta"] is not None:
        res["dbeta"] = db.view(shape)
    if s["bias"] is not None:
        res["dbias"], res["dscale"] = dbias, dscale
    if s["h0"] is not None:
        res["dh0"] = torch.zeros(s["h0"].shape, device=dev, dtype=torch.double) if s["dhT"] is None else \
            s["dhT"].double().clone()
        res["dh0"][rows] = c
    return res


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("step", "scan", "train"):
        return _exact_recurrence(s)
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
        coef = min(1.0, s["max_norm"] / (norm + EPS))
        return {"norm": torch.tensor([norm], dtype=torch.double),
                "out": [g.double() * coef for g in _first_and_last(s["grads"])]}
    x, w = s["x"].double(), s["weight"].double()
    r = x if s["residual"] is None else x + s["residual"].double()
    ms = (r * r).sum(1, keepdim=True) / r.shape[1]
    y = r / torch.sqrt(ms + EPS) * w
    if op == "norm":
        D, g = case["dim"], case["group"] or case["dim"]
        peak = torch.stack([p.abs().amax(1) for p in y.split(g, dim=1)], 1)
        scale = torch.clamp(peak, min=AMAX_FLOOR) / E4M3_MAX
        q = y / scale.repeat_interleave(g, dim=1)[:, :D]
        return {"out": q, "scales": scale if case["group"] else scale[:, 0],
                "residual": None if s["residual"] is None else r}
    res = r.to(s["residual"].dtype).double()  # the gradient is taken at the residual as it is kept
    xhat = res / torch.sqrt(ms + EPS)
    dxhat = s["dy"].double() * w
    dr = (dxhat - xhat * (dxhat * xhat).sum(1, keepdim=True) / r.shape[1]) / torch.sqrt(ms + EPS) + s["dres"].double()
    return {"out": y, "residual": r, "dr": dr, "dweight": (s["dy"].double() * xhat).sum(0)}
