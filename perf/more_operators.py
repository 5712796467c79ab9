"""Cases of the feed-forward and optimizer operators: what a pass reads and returns, its plain form, and its 64-bit value.

Three operators that a block of a recurrent stack has beside its recurrence and its norm, as it is served and trained:

  glu    gdn_glu                       the gated half of a feed-forward block: both projections, the activation, the product
  train  gdn_glu + gdn_glu_backward    a training pass through it
  adamw  gdn_adamw                     the optimizer's step over many tensors, its states in 32 bits or in 8

gdn_glu: g = x w_gate^T, u = x w_up^T, out = act(g) u; its gradient: d_g = d_out u act'(g), d_u = d_out act(g),
dx = d_g w_gate + d_u w_up, d_w_gate = d_g^T x, d_w_up = d_u^T x.

gdn_adamw: k = min(1, max_norm / (norm + 1e-6)) where a norm is given, else 1; m = b1 m + (1 - b1) k g;
v = b2 v + (1 - b2) (k g)^2; p = p - lr (wd p + m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps)).  In 8 bits m and the
root of v are kept in e4m3, by blocks of 256 elements, in units of a 448th of the block's largest (taken as 2^-100 at
least); a root above zero is kept as the smallest e4m3 value at least.

`own` False: elementary torch operations in 32 bits, rounded once at the end.  True: the calls of the package.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SZ = {"f32": 4, "f16": 2, "bf16": 2}
E4M3 = torch.float8_e4m3fn
E4M3_MAX, E4M3_MIN, AMAX_FLOOR = 448.0, 2.0 ** -9, 2.0 ** -100
BLOCK = 256
CLIP_EPS = 1e-6
ACTIVATIONS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest serving call: one request's token, the layer width of 16 heads of 128, an inner width of three times it
        {"name": "glu-1", "op": "glu", "tokens": 1, "dim": 2048, "inner": 6144, "dtype": "f16", "act": "silu"},
        # eight requests' tokens at the width of 32 heads of 128
        {"name": "glu-8", "op": "glu", "tokens": 8, "dim": 4096, "inner": 8192, "dtype": "bf16", "act": "silu"},
        # the decode batch: 256 requests' tokens
        {"name": "glu-256", "op": "glu", "tokens": 256, "dim": 4096, "inner": 8192, "dtype": "f16", "act": "silu"},
        # a small ragged prefill of odd sizes
        {"name": "glu-odd", "op": "glu", "tokens": 1001, "dim": 517, "inner": 1531, "dtype": "f16", "act": "gelu_tanh"},
        # the ragged prefill: 16384 tokens together
        {"name": "glu-prefill", "op": "glu", "tokens": 16384, "dim": 2048, "inner": 6144, "dtype": "bf16", "act": "silu"},
        # a training pass over odd sizes
        {"name": "train-odd", "op": "train", "tokens": 999, "dim": 1000, "inner": 2667, "dtype": "f16", "act": "gelu"},
        # a training pass of a narrow layer over long sequences: few weights, many tokens
        {"name": "train-narrow", "op": "train", "tokens": 32768, "dim": 512, "inner": 1536, "dtype": "bf16",
         "act": "silu"},
        # a training pass over two sequences of 8192 tokens, 16 heads of 128
        {"name": "train-long", "op": "train", "tokens": 16384, "dim": 2048, "inner": 6144, "dtype": "bf16",
         "act": "silu"},
        # one small layer of odd widths, all in 32 bits
        {"name": "adamw-layer", "op": "adamw", "layers": 1, "width": 517, "dtype": "f32", "grad": "f32", "master": False,
         "state": 32, "clip": False},
        # 24 layers of width 2048: 16-bit weights with 32-bit master copies, gradients clipped as they are read
        {"name": "adamw-model", "op": "adamw", "layers": 24, "width": 2048, "dtype": "bf16", "grad": "bf16",
         "master": True, "state": 32, "clip": True},
        # the small layer with 8-bit states
        {"name": "adamw8-layer", "op": "adamw", "layers": 1, "width": 517, "dtype": "f32", "grad": "f16",
         "master": False, "state": 8, "clip": True},
        # 24 layers of width 2048, 16-bit weights and gradients, 8-bit states
        {"name": "adamw8-model", "op": "adamw", "layers": 24, "width": 2048, "dtype": "bf16", "grad": "bf16",
         "master": False, "state": 8, "clip": True},
    ]


MOST_PRODUCT = 16384 * 2048 * 6144  # tokens x dim x inner of the largest pass


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A multiple of 128 half the time, of 8 a quarter, any number otherwise."""
    d = _log(rng, lo, hi)
    by = rng.choice([128, 128, 8, 1])
    return max(by, d // by * by)


def draw(rng):
    op = rng.choice(["glu", "train", "adamw"])
    if op == "adamw":
        width = _log(rng, 100, 2048)
        dtype = rng.choice(["f32", "f16", "bf16"])
        return {"op": op, "layers": _log(rng, 1, max(1, min(24, 24 * 2048 ** 2 // (2 * width ** 2)))), "width": width,
                "dtype": dtype, "grad": rng.choice([dtype, dtype, "f32", "bf16"]),
                "master": dtype != "f32" and rng.random() < 0.5, "state": rng.choice([8, 32]),
                "clip": rng.random() < 0.6}
    dim, inner = _width(rng, 200, 5000), _width(rng, 300, 10000)
    tokens = min(_log(rng, 1 if op == "glu" else 64, 32768), MOST_PRODUCT // (dim * inner))
    return {"op": op, "tokens": tokens, "dim": dim, "inner": inner, "dtype": rng.choice(["f16", "bf16"]),
            "act": rng.choice(["silu", "silu"] + list(ACTIVATIONS[1:]))}


# ------------------------------------------------------------------ inputs
def _sizes(case):
    """The weights of a stack of recurrent blocks: projections, gate parameters, norm weights."""
    w = case["width"]
    return [(w, w), (w, w), (w, w), (w, w), (w,), (w,), (w,)] * case["layers"]


def _quantised(y):
    """Blocks [n, 256] in e4m3, and the scales [n]."""
    scale = torch.clamp(y.abs().amax(1), min=AMAX_FLOOR) / E4M3_MAX
    q = y / scale[:, None]
    return q, scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    if case["op"] != "adamw":
        T, D, F, dt = case["tokens"], case["dim"], case["inner"], DT[case["dtype"]]
        # rows of a normed stream, projections that keep its variance
        s = {"case": case, "x": normal(T, D, dtype=dt), "w_gate": normal(F, D, std=D ** -0.5, dtype=dt),
             "w_up": normal(F, D, std=D ** -0.5, dtype=dt)}
        if case["op"] == "train":
            s["d_out"] = normal(T, F, dtype=dt)
        else:
            s["out"] = torch.zeros(T, F, dtype=dt, device=dev)
        return s

    # the tensors are parts of flat buffers, each from a multiple of 256 elements on; what is between them stays zero
    shapes = _sizes(case)
    spans, n = [], 0
    for shape in shapes:
        spans.append((n, math.prod(shape), shape))
        n += -(-math.prod(shape) // BLOCK) * BLOCK
    used = torch.zeros(n, dtype=torch.bool, device=dev)
    for at, size, _ in spans:
        used[at:at + size] = True
    keep = lambda t: t * used  # noqa: E731

    def parts(flat, dtype=None):
        return [flat[at:at + size].view(shape) for at, size, shape in spans]

    p = keep(normal(n, std=0.02))
    m = keep(normal(n, std=1e-4))
    v = keep(normal(n, std=1e-3)).square()
    s = {"case": case, "grad": keep(normal(n, std=1e-3, dtype=DT[case["grad"]]).float()).to(DT[case["grad"]]),
         "param": p.to(DT[case["dtype"]]), "master": p if case["master"] else None, "step": 100 + int(seed) % 50}
    s["norm"] = torch.full((1,), 1e-3 * math.sqrt(n), device=dev) if case["clip"] else None
    s["max_norm"] = 0.5e-3 * math.sqrt(n) if case["clip"] else None
    if case["state"] == 8:
        for name, y in (("exp_avg", m), ("exp_avg_sq", v.sqrt())):
            q, scale = _quantised(y.view(-1, BLOCK))
            s[name], s[name + "_scales"] = q.to(E4M3).view(-1), scale
    else:
        s["exp_avg"], s["exp_avg_sq"] = m, v
    for name in ("grad", "param", "master", "exp_avg", "exp_avg_sq"):
        s[name + "s"] = None if s[name] is None else parts(s[name])
    for name in ("exp_avg_scales", "exp_avg_sq_scales"):
        s[name + "_list"] = None if name not in s else [s[name][at // BLOCK:at // BLOCK + -(-size // BLOCK)]
                                                        for at, size, _ in spans]
    s["hyper"] = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}
    return s


# ------------------------------------------------------------------ plain forms, 32 bits
def _act(g, kind):
    """act(g) and act'(g)."""
    if kind in ("silu", "sigmoid"):
        s = 1 / (1 + torch.exp(-g))
        return (s, s * (1 - s)) if kind == "sigmoid" else (g * s, s * (1 + g * (1 - s)))
    if kind == "relu":
        return torch.clamp(g, min=0), (g > 0).to(g.dtype)
    if kind == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _plain_glu(s):
    dt, kind = s["x"].dtype, s["case"]["act"]
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    g, u = x @ wg.T, x @ wu.T
    a, slope = _act(g, kind)
    if s["case"]["op"] == "glu":
        s["out"].copy_(a * u)
        return {"out": s["out"]}
    d = s["d_out"].float()
    dg, du = d * u * slope, d * a
    return {"out": (a * u).to(dt), "dx": (dg @ wg + du @ wu).to(dt), "d_w_gate": (dg.T @ x).to(dt),
            "d_w_up": (du.T @ x).to(dt)}


def _plain_adamw(s):
    h, t = s["hyper"], s["step"]
    g = s["grad"].float()
    if s["norm"] is not None:
        g = g * torch.clamp(s["max_norm"] / (s["norm"] + CLIP_EPS), max=1.0)
    p = s["param"].float() if s["master"] is None else s["master"]
    m, v = s["exp_avg"], s["exp_avg_sq"]
    if s["case"]["state"] == 8:
        m = (m.float().view(-1, BLOCK) * s["exp_avg_scales"][:, None]).view(-1)
        v = (v.float().view(-1, BLOCK) * s["exp_avg_sq_scales"][:, None]).square().view(-1)
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g.square()
    c1, c2 = 1 - h["beta1"] ** t, 1 - h["beta2"] ** t
    p = p - h["lr"] * (h["weight_decay"] * p + m / c1 / (torch.sqrt(v / c2) + h["eps"]))
    s["param"].copy_(p)
    out = {"param": s["param"]}
    if s["master"] is not None:
        s["master"].copy_(p)
        out["master"] = s["master"]
    if s["case"]["state"] == 8:
        q, scale = _quantised(m.view(-1, BLOCK))
        s["exp_avg"].copy_(q.view(-1).to(E4M3))
        s["exp_avg_scales"].copy_(scale)
        q, scale = _quantised(torch.sqrt(v).view(-1, BLOCK))
        q = torch.where(q > 0, torch.clamp(q, min=E4M3_MIN), q)
        s["exp_avg_sq"].copy_(q.view(-1).to(E4M3))
        s["exp_avg_sq_scales"].copy_(scale)
        out |= {"exp_avg_scales": s["exp_avg_scales"], "exp_avg_sq_scales": s["exp_avg_sq_scales"]}
    else:
        s["exp_avg"].copy_(m)
        s["exp_avg_sq"].copy_(v)
    return out | {"exp_avg": s["exp_avg"], "exp_avg_sq": s["exp_avg_sq"]}


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import gated_delta_rule_gate_gb300 as gdn
    case = s["case"]
    if case["op"] == "glu":
        gdn.gdn_glu(s["x"], s["w_gate"], s["w_up"], activation=case["act"], out=s["out"])
        return {"out": s["out"]}
    if case["op"] == "train":
        out, gates = gdn.gdn_glu(s["x"], s["w_gate"], s["w_up"], activation=case["act"], want_gates=True)
        b = gdn.gdn_glu_backward(s["d_out"], s["x"], s["w_gate"], s["w_up"], gates, activation=case["act"])
        return {"out": out, "dx": b.dx, "d_w_gate": b.d_w_gate, "d_w_up": b.d_w_up}
    gdn.gdn_adamw(s["params"], s["grads"], s["exp_avgs"], s["exp_avg_sqs"], s["step"], master=s["masters"],
                  exp_avg_scales=s["exp_avg_scales_list"], exp_avg_sq_scales=s["exp_avg_sq_scales_list"],
                  grad_norm=s["norm"], max_norm=s["max_norm"], **s["hyper"])
    return {k: s[k] for k in ("param", "master", "exp_avg", "exp_avg_sq", "exp_avg_scales", "exp_avg_sq_scales")
            if s.get(k) is not None}


def run(state):
    if own:
        return _own(state)
    return _plain_adamw(state) if state["case"]["op"] == "adamw" else _plain_glu(state)


# ------------------------------------------------------------------ work
def work(case):
    e = SZ[case["dtype"]]
    if case["op"] == "adamw":
        n = sum(math.prod(s) for s in _sizes(case))
        states = 4 * 4 if case["state"] == 32 else 4
        scales = 0 if case["state"] == 32 else 4 * 4 * sum(-(-math.prod(s) // BLOCK) for s in _sizes(case))
        # gradient in; weight in and out, or the master copy in and out and the weight out; both states in and out
        weights = 2 * e if not case["master"] else 8 + e
        return {"bytes": n * (SZ[case["grad"]] + weights + states) + scales, "flops": 16 * n}
    T, D, F = case["tokens"], case["dim"], case["inner"]
    if case["op"] == "glu":
        return {"bytes": e * (T * D + 2 * F * D + T * F), "flops": 4 * T * D * F + 8 * T * F}
    # x, weights, d_out in; out, dx and the weights' gradients out; three products of the size of the forward pass's
    return {"bytes": e * (2 * T * D + 4 * F * D + 2 * T * F), "flops": 12 * T * D * F + 24 * T * F}


# ------------------------------------------------------------------ 64 bits
def _exact_activation(g, kind):
    """act and its derivative in 64 bits by the functions' own definitions."""
    one = torch.ones_like(g)
    sig = torch.sigmoid(g)
    if kind == "silu":
        return g * sig, sig + g * sig * (one - sig)
    if kind == "sigmoid":
        return sig, sig * (one - sig)
    if kind == "relu":
        return torch.where(g > 0, g, 0 * one), torch.where(g > 0, one, 0 * one)
    if kind == "gelu":
        phi = torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        normal = torch.special.ndtr(g)
        return g * normal, normal + g * phi
    inner = math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)
    # (1 + tanh z) / 2 = sigmoid(2 z)
    half = torch.sigmoid(2 * inner)
    return g * half, half + g * 2 * half * (one - half) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "adamw":
        x, wg, wu = s["x"].double(), s["w_gate"].double(), s["w_up"].double()
        g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        a, slope = _exact_activation(g, case["act"])
        if case["op"] == "glu":
            return {"out": a * u}
        d = s["d_out"].double()
        du, dg = d * a, d * u * slope
        dx = torch.mm(dg, wg).add_(torch.mm(du, wu))
        return {"out": a * u, "dx": dx, "d_w_gate": torch.mm(dg.t(), x), "d_w_up": torch.mm(du.t(), x)}
    h, t = s["hyper"], s["step"]
    k = 1.0 if s["norm"] is None else min(1.0, s["max_norm"] / (float(s["norm"]) + CLIP_EPS))
    g = s["grad"].double() * k
    eight = case["state"] == 8
    m, r = s["exp_avg"].to(torch.float32).double(), s["exp_avg_sq"].to(torch.float32).double()
    if eight:
        m *= s["exp_avg_scales"].double().repeat_interleave(BLOCK)
        r *= s["exp_avg_sq_scales"].double().repeat_interleave(BLOCK)
        v = r * r
    else:
        v = r
    m = torch.lerp(g, m, h["beta1"])
    v = torch.lerp(g * g, v, h["beta2"])
    rate = h["lr"] / -math.expm1(t * math.log(h["beta1"]))
    root = torch.sqrt(v)
    denom = root / math.sqrt(-math.expm1(t * math.log(h["beta2"]))) + h["eps"]
    old = (s["master"] if s["master"] is not None else s["param"]).double()
    p = old * (1 - h["lr"] * h["weight_decay"]) - rate * m / denom
    out = {"param": p, "exp_avg": m, "exp_avg_sq": v}
    if s["master"] is not None:
        out["master"] = p
    if eight:
        for name, y in (("exp_avg", m), ("exp_avg_sq", root)):
            scale = torch.clamp(y.abs().view(-1, BLOCK).amax(1), min=AMAX_FLOOR) / E4M3_MAX
            q = y / scale.repeat_interleave(BLOCK)
            out[name] = q if name == "exp_avg" else torch.where(q > 0, torch.clamp(q, min=E4M3_MIN), q)
            out[name + "_scales"] = scale
    return out
