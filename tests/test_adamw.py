"""gdn_adamw against the formula in 64 bits, and its refusals.

Tolerances (u = 2^-24, a rounding of fp32).  m is two products and a sum of values that
carry the clip factor's error: within 8 u of |beta1 m| + |(1 - beta1) k g|, which is called
M.  v likewise, with the square of the factor: 16 u.  The root of v halves that, and with
its own rounding, the bias corrections (expm1f: 2 ulp) and the divisions the step lr m /
(...) is within 64 u of what M in place of m would give.  p adds two roundings of its own,
and one of its type.  An 8-bit code is the quotient by its scale, off by half a step of e4m3
(2^-4 of the value, 2^-10 below 2^-6) and by what m or the root itself is off.
"""
import ctypes
import math

import pytest
import torch

import layer_reference as ref
from gated_delta_rule_gate_gb300 import _native as N

U = 2.0 ** -24
FAKE = 0x100000
BLOCK = 256
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


class Case:
    """Tensors of a step on the GPU, and what they were before."""

    def __init__(self, seed, sizes, types=("f32",), grads=("f32",), eight=False, master=False, fresh=False, at=0):
        gen = torch.Generator().manual_seed(seed)

        def place(v, dtype):
            # `at` elements behind a 512-byte address
            flat = torch.zeros(v.numel() + at, dtype=dtype, device="cuda")
            flat[at:] = v.to(dtype).cuda()
            return flat[at:]

        draw = lambda n, std: torch.randn(n, generator=gen) * std
        self.p, self.g, self.m, self.v, self.ms, self.vs, self.w = [], [], [], [], [], [], []
        for i, n in enumerate(sizes):
            dt = ref.DT[types[i % len(types)]]
            p = draw(n, 0.5)
            self.p.append(place(p, dt))
            self.w.append(place(p + draw(n, 1e-4), torch.float32) if master and dt != torch.float32 else None)
            self.g.append(place(draw(n, 0.1), ref.DT[grads[i % len(grads)]]))
            m, r = draw(n, 0.05), draw(n, 0.1).abs()
            if fresh:
                m, r = m * 0, r * 0
            if eight:
                nb = -(-n // BLOCK)
                for y, codes, scales in ((m, self.m, self.ms), (r, self.v, self.vs)):
                    pad = torch.zeros(nb * BLOCK)
                    pad[:n] = y
                    s = pad.view(nb, BLOCK).abs().amax(1) / 448 if nb else torch.zeros(0)
                    q = torch.where(s[:, None] > 0, pad.view(nb, BLOCK) / s[:, None], torch.zeros(1))
                    codes.append(place(q.reshape(-1)[:n].to(torch.float8_e4m3fn).float(), torch.float8_e4m3fn))
                    scales.append(s.cuda())
            else:
                self.m.append(place(m, torch.float32))
                self.v.append(place(r * r, torch.float32))
        self.eight = eight
        self.before = {k: [None if t is None else t.clone() for t in getattr(self, k)]
                       for k in ("p", "g", "m", "v", "ms", "vs", "w")}

    def lists(self):
        more = dict(exp_avg_scales=self.ms, exp_avg_sq_scales=self.vs) if self.eight else {}
        if any(t is not None for t in self.w):
            more["master"] = self.w
        return (self.p, self.g, self.m, self.v), more

    def tensors(self):
        return [t for k in ("p", "m", "v", "ms", "vs", "w") for t in getattr(self, k) if t is not None]

    def run(self, step=7, **kw):
        import gated_delta_rule_gate_gb300 as g
        lists, more = self.lists()
        assert g.gdn_adamw(*lists, step, **{**HYPER, **more, **kw}) is None
        return self

    def check(self, t=7, k=1.0, **kw):
        h = {**HYPER, **kw}
        b = self.before
        for i in range(len(self.p)):
            assert torch.equal(self.g[i], b["g"][i])
            n = self.p[i].numel()
            if n == 0:
                continue
            p = (b["p"][i] if b["w"][i] is None else b["w"][i]).double()
            g = b["g"][i].double() * k
            m, v = b["m"][i].double(), b["v"][i].double()
            if self.eight:
                m = m * b["ms"][i].double().repeat_interleave(BLOCK)[:n]
                v = (v * b["vs"][i].double().repeat_interleave(BLOCK)[:n]) ** 2
            M = (h["beta1"] * m).abs() + ((1 - h["beta1"]) * g).abs()
            m = h["beta1"] * m + (1 - h["beta1"]) * g
            v = h["beta2"] * v + (1 - h["beta2"]) * g * g
            rate = h["lr"] / (1 - h["beta1"] ** t)
            den = v.sqrt() / math.sqrt(1 - h["beta2"] ** t) + h["eps"]
            want = p - h["lr"] * h["weight_decay"] * p - rate * m / den
            tol = 4 * U * (p.abs() + want.abs()) + 64 * U * rate * M / den + 1e-37
            if self.w[i] is not None:
                assert bool(((self.w[i].double() - want).abs() <= tol).all())
            tiny = 2.0 ** -25 if self.p[i].dtype == torch.float16 else 0.0
            r = ref.ROUND[self.p[i].dtype]
            assert bool(((self.p[i].double() - want).abs() <= (1 + r) * tol + r * want.abs() + tiny).all())
            if not self.eight:
                assert bool(((self.m[i].double() - m).abs() <= 8 * U * M + 1e-37).all())
                assert bool(((self.v[i].double() - v).abs() <= 16 * U * v + 1e-37).all())
                continue
            for y, err, codes, scales in ((m, 8 * U * M, self.m[i], self.ms[i]),
                                          (v.sqrt(), 16 * U * v.sqrt(), self.v[i], self.vs[i])):
                nb = -(-n // BLOCK)
                pad = torch.zeros(nb * BLOCK, dtype=torch.double, device="cuda")
                pad[:n] = y.abs()
                s = pad.view(nb, BLOCK).amax(1).clamp(min=2.0 ** -100) / 448
                off = torch.zeros_like(pad)
                off[:n] = err
                assert bool(((scales.double() - s).abs() <= off.view(nb, BLOCK).amax(1) / 448 + 4 * U * s).all())
                s = s.repeat_interleave(BLOCK)[:n]
                q = y / s
                if codes is self.v[i]:
                    q = torch.where(q > 0, q.clamp(min=2.0 ** -9), q)
                worst = off.max() / s + 8 * U * q.abs()
                assert bool(((codes.double() - q).abs() <= (q.abs() + worst) * 2.0 ** -4 + 2.0 ** -10 + worst).all())


LISTS = [
    ([1], ("f32",), ("f32",)),
    ([0, 5, 0], ("f16",), ("f16",)),
    ([255, 256, 257, 3], ("bf16", "f32"), ("bf16", "f32")),
    ([100000, 1, 17, 65536, 12345], ("f32", "f16", "bf16"), ("f32", "bf16")),
    ([300 + i for i in range(33)], ("f32", "bf16"), ("f16",)),
    ([64 + i % 7 for i in range(1000)], ("f16", "f32", "bf16"), ("f16", "f32")),
    ([70 + i % 300 for i in range(900)], ("bf16",), ("f32",)),  # several tables of one kind
    ([5000001], ("f32",), ("f32",)),
    ([9000000, 7], ("bf16",), ("bf16",)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("i", range(len(LISTS)))
def test_matches_the_formula(i, eight, master):
    Case(i, *LISTS[i], eight=eight, master=master).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_any_address(eight):
    """Every offset from a word's address, shorter than a group of four and longer."""
    for n in (1, 3, 4, 5, 127, 700):
        for at in range(1, 8):
            for dt in ("f32", "bf16"):
                Case(n + at, [n], (dt,), ("f16",), eight=eight, master=True, at=at).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_parts_of_flat_buffers(eight):
    """What lies between the tensors is left alone."""
    import gated_delta_rule_gate_gb300 as g
    gen = torch.Generator().manual_seed(4)
    state = torch.float8_e4m3fn if eight else torch.float32
    flats = [torch.randn(5000, generator=gen).abs().to(dt).cuda() for dt in (torch.float32, state, state)]
    grad = torch.randn(5000, generator=gen).cuda()
    before = [t.clone() for t in flats]
    spans = [(1, 9), (512, 1536), (1537, 1537), (2001, 4003)]
    cut = lambda t: [t[a:b] for a, b in spans]
    scales = [[torch.ones(-(-(b - a) // BLOCK), device="cuda") for a, b in spans] for _ in range(2)]
    more = dict(exp_avg_scales=scales[0], exp_avg_sq_scales=scales[1]) if eight else {}
    g.gdn_adamw(cut(flats[0]), cut(grad), cut(flats[1]), cut(flats[2]), 1, **more)
    for t, b in zip(flats, before):
        for a, e in ((0, 1), (9, 512), (1536, 2001), (4003, 5000)):
            assert torch.equal(t[a:e].float(), b[a:e].float())
        assert not torch.equal(t[2001:4003].float(), b[2001:4003].float())


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_first_step_and_large_numbers(eight):
    """Zero states; the corrections of the first step and of a late one; betas of zero."""
    for step in (1, 2, 1000, 2 ** 31 - 1):
        Case(step % 97, [1000], eight=eight, fresh=True).run(step).check(step)
    Case(5, [1000], eight=eight).run(3, beta1=0.0, beta2=0.0).check(3, beta1=0.0, beta2=0.0)
    Case(6, [1000], eight=eight).run(3, lr=0.0).check(3, lr=0.0)
    Case(7, [1000], eight=eight).run(3, beta2=0.99999).check(3, beta2=0.99999)


@pytest.mark.gpu
def test_codes_are_those_of_the_formula_in_fp32():
    """Each operation rounded to fp32 in its turn gives the same codes and scales, to the bit,
    over several steps: none of 2 million values is on the wrong side of a border."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    n = 1 << 21
    c = Case(21, [n], ("f32",), ("f32",), eight=True)
    m, v, ms, vs = (t[0].clone() for t in (c.m, c.v, c.ms, c.vs))
    norm = torch.tensor([3.7], device="cuda")
    for step in (1, 2, 50):
        c.g[0].copy_(torch.randn(n, generator=gen, device="cuda") * 10.0 ** (torch.arange(n, device="cuda") % 7 - 5))
        c.run(step, grad_norm=norm, max_norm=1.3)
        g = c.g[0] * torch.clamp(1.3 / (norm + 1e-6), max=1.0)
        m32 = (m.float().view(-1, BLOCK) * ms[:, None]).view(-1)
        v32 = (v.float().view(-1, BLOCK) * vs[:, None]).square().view(-1)
        m32 = HYPER["beta1"] * m32 + (1 - HYPER["beta1"]) * g
        v32 = HYPER["beta2"] * v32 + (1 - HYPER["beta2"]) * g.square()
        new = []
        for y in (m32, torch.sqrt(v32)):
            y = y.view(-1, BLOCK)
            s = torch.clamp(y.abs().amax(1), min=2.0 ** -100) * (1 / 448)
            q = y / s[:, None]
            if new:
                q = torch.where(q > 0, torch.clamp(q, min=2.0 ** -9), q)
            new += [q.view(-1).to(torch.float8_e4m3fn), s]
        m, ms, v, vs = new
        for a, b in ((c.m[0], m), (c.ms[0], ms), (c.v[0], v), (c.vs[0], vs)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.gpu
def test_zero_gradients_keep_zero_states():
    for eight in (False, True):
        c = Case(3, [700, 20], eight=eight, fresh=True)
        for g in c.g:
            g.zero_()
        c.before["g"] = [g.clone() for g in c.g]
        c.run(1).check(1)
        assert not any(bool(t.float().any()) for t in c.m + c.v)


@pytest.mark.gpu
def test_a_small_root_keeps_a_code():
    """A gradient far below its block's largest divides by no less than the smallest code."""
    c = Case(3, [300], eight=True, fresh=True)
    c.g[0].fill_(1e-9)
    c.g[0][5] = 10.0
    c.before["g"] = [c.g[0].clone()]
    c.run(1).check(1)
    v = c.v[0].float()
    assert float(v[5]) == 448 and bool((v[:256][torch.arange(256) != 5] == 2.0 ** -9).all())


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_step_rate_and_norm_on_the_device(eight):
    step = torch.tensor([12], dtype=torch.int64, device="cuda")
    lr = torch.tensor(0.02, device="cuda")
    c = Case(8, [3000, 11], ("bf16", "f32"), eight=eight, master=True)
    norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in c.g))
    at = torch.tensor([norm], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.run(step, lr=lr, grad_norm=at, max_norm=0.4 * norm, error_word=err)
    c.check(12, k=0.4 * norm / (float(at) + 1e-6), lr=float(lr))
    assert int(err) == 0
    c = Case(8, [3000, 11], eight=eight)
    c.run(step, grad_norm=at, max_norm=2 * norm).check(12)  # in bounds


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_a_norm_that_is_not_finite_takes_no_step(bad):
    for eight in (False, True):
        c = Case(9, [1000, 77], ("bf16",), eight=eight, master=True)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.run(grad_norm=torch.tensor([bad], device="cuda"), max_norm=1.0, error_word=err)
        assert int(err) == N.DEVERR_NONFINITE
        for k in ("p", "m", "v", "ms", "vs", "w"):
            assert all(a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                       for a, b in zip(getattr(c, k), c.before[k]))


@pytest.mark.gpu
def test_clip_norm_and_step_together():
    """gdn_grad_clip's norm, without scaling, then the step that clips as it reads, equals the
    gradients clipped first to within the rounding that this saves."""
    import gated_delta_rule_gate_gb300 as g
    c, d = Case(10, [4000, 130]), Case(10, [4000, 130])
    old = [t.clone() for t in c.g]
    norm = g.gdn_grad_clip(c.g, 3e38)
    assert all(torch.equal(a, b) for a, b in zip(c.g, old))
    c.run(grad_norm=norm, max_norm=0.1).check(k=0.1 / (float(norm) + 1e-6))
    g.gdn_grad_clip(d.g, 0.1)
    d.run()
    for a, b in zip(c.p, d.p):
        assert bool(((a - b).abs() <= 1e-5 * HYPER["lr"] + 4 * U * a.abs()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_captured_steps_equal_eager_ones(eight):
    """A graph of the norm and the step, replayed with a step number that it counts up itself."""
    import gated_delta_rule_gate_gb300 as g
    a, b = (Case(11, [9000, 65], ("bf16",), ("bf16",), eight=eight, master=True, fresh=True) for _ in range(2))
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g.gdn_grad_clip(a.g, 3e38)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        a.run(step, grad_norm=g.gdn_grad_clip(a.g, 3e38), max_norm=1.0)
    one = torch.zeros(1, dtype=torch.int64, device="cuda")
    for _ in range(4):
        graph.replay()
        one.add_(1)
        b.run(one, grad_norm=g.gdn_grad_clip(b.g, 3e38), max_norm=1.0)
    torch.cuda.synchronize()
    assert int(step) == 4
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.tensors(), b.tensors()))


@pytest.mark.gpu
def test_a_copy_of_an_fp32_parameter():
    """It is the copy that the step is taken on; the parameter receives it."""
    for eight in (False, True):
        c = Case(14, [700, 30], ("f32",), ("bf16",), eight=eight)
        c.w = [p + 0.25 for p in c.p]
        c.before["w"] = [w.clone() for w in c.w]
        c.p[0].fill_(float("nan"))
        c.run().check()
        assert all(torch.equal(p, w) for p, w in zip(c.p, c.w))


@pytest.mark.gpu
def test_empty_lists():
    import gated_delta_rule_gate_gb300 as g
    assert g.gdn_adamw([], [], [], [], 1) is None
    e = torch.zeros(0, device="cuda")
    assert g.gdn_adamw([e], [e], [e], [e], 1) is None


@pytest.mark.gpu
def test_on_another_stream():
    c = Case(12, [200000, 3], ("bf16", "f32"), eight=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    c.check()


@pytest.mark.gpu
def test_autograd_notices_the_step():
    c = Case(13, [50])
    p = c.p[0]
    saved = p._version
    c.run()
    assert p._version > saved and c.g[0]._version == Case(13, [50]).g[0]._version


# ---------------------------------------------------------------- refusals (no GPU)
def _args(n=2, **over):
    vp = ctypes.c_void_p * n
    ptr = lambda values: vp(*values)
    a = N.GdnAdamwArgs()
    a.count, a.state_dtype, a.step = n, N.DTYPE_F32, 1
    a.lr, a.beta1, a.beta2, a.eps, a.weight_decay, a.norm_eps = 1e-3, 0.9, 0.999, 1e-8, 0.01, 1e-6
    keep = {k: ptr(over.pop(k, [FAKE] * n)) for k in ("params", "grads", "exp_avg", "exp_avg_sq")}
    for k in ("exp_avg_scales", "exp_avg_sq_scales", "master"):
        if k in over:
            keep[k] = ptr(over.pop(k))
    keep["sizes"] = (ctypes.c_int64 * n)(*over.pop("sizes", [4] * n))
    for k, d in (("param_dtypes", [0, 1]), ("grad_dtypes", [2, 0])):
        keep[k] = (ctypes.c_int32 * n)(*over.pop(k, d[:n]))
    for k, v in keep.items():
        setattr(a, k, ctypes.cast(v, dict(N.GdnAdamwArgs._fields_)[k]))
    for k, v in over.items():
        setattr(a, k, v)
    a._keep = keep
    return a


@pytest.mark.parametrize("over,status,msg", [
    (dict(count=-1), N.GDN_ERR_INVALID, "count"),
    (dict(state_dtype=1), N.GDN_ERR_INVALID, "state_dtype"),
    (dict(step=0), N.GDN_ERR_INVALID, "step"),
    (dict(lr=-1.0), N.GDN_ERR_INVALID, "lr"),
    (dict(lr=math.nan), N.GDN_ERR_INVALID, "lr"),
    (dict(beta1=1.0), N.GDN_ERR_INVALID, "beta1"),
    (dict(beta2=-0.1), N.GDN_ERR_INVALID, "beta2"),
    (dict(beta2=math.nan), N.GDN_ERR_INVALID, "beta2"),
    (dict(eps=-1e-8), N.GDN_ERR_INVALID, "eps"),
    (dict(weight_decay=math.inf), N.GDN_ERR_INVALID, "weight_decay"),
    (dict(grad_norm=FAKE, max_norm=-1.0), N.GDN_ERR_INVALID, "max_norm"),
    (dict(grad_norm=FAKE, max_norm=1.0, norm_eps=math.nan), N.GDN_ERR_INVALID, "norm_eps"),
    (dict(param_dtypes=[0, 3]), N.GDN_ERR_INVALID, "tensor 1"),
    (dict(grad_dtypes=[4, 0]), N.GDN_ERR_INVALID, "tensor 0"),
    (dict(sizes=[-1, 4]), N.GDN_ERR_INVALID, "tensor 0"),
    (dict(sizes=[(1 << 40) + 1, 4]), N.GDN_ERR_UNSUPPORTED, "2^40"),
    (dict(params=[FAKE, None]), N.GDN_ERR_INVALID, "tensor 1"),
    (dict(exp_avg_sq=[None, FAKE]), N.GDN_ERR_INVALID, "tensor 0"),
    (dict(grads=[FAKE + 1, FAKE]), N.GDN_ERR_INVALID, "aligned"),
    (dict(exp_avg=[FAKE + 2, FAKE]), N.GDN_ERR_INVALID, "aligned"),
    (dict(master=[FAKE + 2, FAKE]), N.GDN_ERR_INVALID, "aligned"),
    (dict(step_device=FAKE + 4), N.GDN_ERR_INVALID, "aligned"),
    (dict(state_dtype=N.DTYPE_E4M3), N.GDN_ERR_INVALID, "scales"),
    (dict(exp_avg_scales=[FAKE, FAKE]), N.GDN_ERR_INVALID, "scales"),
    (dict(state_dtype=N.DTYPE_E4M3, exp_avg_scales=[FAKE, FAKE], exp_avg_sq_scales=[FAKE, None]), N.GDN_ERR_INVALID,
     "tensor 1"),
])
def test_refuses(over, status, msg):
    a = _args(**over)
    lib = N.load()
    assert lib.gdn_adamw(ctypes.byref(a), None) == status
    assert msg.lower() in N.last_error_message().lower()
    assert lib.gdn_adamw(None, None) == N.GDN_ERR_INVALID


def test_binding_refuses():
    import gated_delta_rule_gate_gb300 as g
    from layer_standins import Standin
    f8 = torch.float8_e4m3fn
    t, u = Standin((4,)), Standin((5,))
    call = g.gdn_adamw
    for args, kw, exc, msg in [
        (([t], [t], [t], [t]), {}, TypeError, "step"),
        (([t], [t], [t], [t], None), {}, TypeError, "step"),
        (([t], [t], [t], [t], 0), {}, ValueError, "step"),
        (([t], [t], [t], [t], 1.5), {}, TypeError, "integer"),
        (([t], [t, t], [t], [t], 1), {}, ValueError, "grads has 2"),
        (([t], [t], [t], [], 1), {}, ValueError, "exp_avg_sq has 0"),
        (([t], [u], [t], [t], 1), {}, ValueError, "gradient must be"),
        (([t], [t], [u], [t], 1), {}, ValueError, "exp_avg must be"),
        (([t], [t], [t], [Standin((4,), dtype=f8)], 1), {}, TypeError, "exp_avg_sq"),
        (([t], [t], [Standin((4,), dtype=torch.float16)], [t], 1), {}, TypeError, "exp_avg"),
        (([t], [t], [t], [t], 1), dict(master=[Standin((4,), dtype=torch.float16)]), TypeError, "master"),
        (([t], [t], [t], [t], 1), dict(grad_norm=Standin((1,))), ValueError, "go together"),
        (([t], [t], [t], [t], 1), dict(max_norm=1.0), ValueError, "go together"),
        (([t], [t], [t], [t], 1), dict(grad_norm=Standin((2,)), max_norm=1.0), ValueError, "one element"),
        (([t], [t], [t], [t], Standin((1,), dtype=torch.int32)), {}, TypeError, "step"),
        (([t], [t], [t], [t], 1), dict(lr=Standin((1,), dtype=torch.float64)), TypeError, "lr"),
        (([Standin((4, 4), (1, 4))], [Standin((4, 4))], [Standin((4, 4))], [Standin((4, 4))], 1), {}, ValueError,
         "contiguous"),
        (([t], [Standin((4,), device="cuda:1")], [t], [t], 1), {}, ValueError, "cuda:1"),
        (([t], [t], [t], [t], Standin((1,), dtype=torch.int64, device="cuda:1")), {}, ValueError, "cuda:1"),
        (([torch.zeros(4)], [torch.zeros(4)], [torch.zeros(4)], [torch.zeros(4)], 1), {}, ValueError, "cpu"),
        (([Standin((600,))], [Standin((600,))], [Standin((600,), dtype=f8)], [Standin((600,), dtype=f8)], 1),
         dict(exp_avg_scales=[Standin((2,))], exp_avg_sq_scales=[Standin((3,))]), ValueError, "exp_avg_scales must be"),
        ((None, [t], [t], [t], 1), {}, TypeError, "params"),
        (([t], [t], [t], [t], 1), dict(betas=1), TypeError, "unexpected"),
    ]:
        with pytest.raises(exc, match=msg):
            call(*args, **kw)
