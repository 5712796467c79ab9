"""gdn_glu and gdn_glu_backward against the formulas in 64 bits, and their refusals.

Tolerances.  A sum of K products is kept in fp32; the tensor cores add 16 products at a
time and may cut where fp32 rounds: each of the K / 16 + 2 additions is within 2^-22 of the sum
of the products' sizes.  An activation is formed in fp32 from an exponential whose argument
is off by 2^-24 of itself: within (8 + |z| + g^2) 2^-22 of its value, z the argument, and its
derivative within four times that of 1 (its terms are of that size).  Kept gates are cut to 24
bits: within 2^-15 of the value.  Results, d_g and
d_u carry a rounding of their type (below fp16's normal numbers 2^-25).  The roundings of d_g and
d_u are independent, so besides the bound on each value the norm of all errors stays within
one rounding of the norm of the result (they add up in squares to less).
"""
import ctypes

import pytest
import torch

import layer_reference as ref
from gated_delta_rule_gate_gb300 import _native as N

FAKE = 0x100000
ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")
ROOT_2_PI = (2 / torch.pi) ** 0.5


def act(g, kind):
    """act(g), act'(g) and the argument of the exponential, 64 bits."""
    if kind == "relu":
        return g.clamp(min=0), (g > 0).double(), g * 0
    if kind == "gelu":
        cdf = torch.special.ndtr(g)
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / (2 * torch.pi) ** 0.5, g
    z = 2 * ROOT_2_PI * (g + 0.044715 * g ** 3) if kind == "gelu_tanh" else g
    s, r = torch.sigmoid(z), torch.sigmoid(-z)
    if kind == "sigmoid":
        return s, s * r, z
    slope = 2 * ROOT_2_PI * (1 + 3 * 0.044715 * g * g) if kind == "gelu_tanh" else 1.0
    return g * s, s + g * s * r * slope, z


def fuzz(g, z):
    return (8 + z.abs() + g * g) * 2.0 ** -22


def tiny(dt):
    return 2.0 ** -25 if dt == torch.float16 else 0.0


def summed(a, b):
    """a @ b of 64-bit matrices and the bound on its fp32 sum."""
    return a @ b, (a.shape[1] / 16 + 2) * 2.0 ** -22 * (a.abs() @ b.abs())


def draw(T, D, F, dt, seed=0, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    d = ref.DT[dt]
    return (r(T, D).to(d).cuda(), (r(F, D) * spread * D ** -0.5).to(d).cuda(), (r(F, D) * D ** -0.5).to(d).cuda(),
            r(T, F).to(d).cuda())


def unpack(gates, F):
    """g and u of kept gates, [rows, 2, F] fp32: the upper halves, and the next bytes by 64 columns."""
    Fg = -(-F // 64) * 64
    assert gates.dtype == torch.uint8 and gates.shape[-1] == 6 * Fg
    rows = gates.reshape(-1, 6 * Fg)
    hi = rows[:, :4 * Fg].contiguous().view(torch.int16).view(-1, 2, Fg).int() << 16
    lo = rows[:, 4 * Fg:].reshape(-1, Fg // 64, 2, 64).transpose(1, 2).reshape(-1, 2, Fg).int() << 8
    return (hi | lo).view(torch.float32)[:, :, :F]


def check_forward(out, gates, x, wg, wu, kind):
    r, t = ref.ROUND[out.dtype], tiny(out.dtype)
    g, eg = summed(x.double(), wg.double().T)
    u, eu = summed(x.double(), wu.double().T)
    a, _, z = act(g, kind)
    want = a * u
    ea = 1.13 * eg + fuzz(g, z) * a.abs()
    tol = ea * u.abs() + a.abs() * eu + ea * eu
    tol = tol + r * (want.abs() + tol) + t
    assert bool(((out.double() - want).abs() <= tol).all())
    if gates is not None:
        kept = unpack(gates, wg.shape[0]).double()
        for k, y, e in ((0, g, eg), (1, u, eu)):
            assert bool(((kept[:, k] - y).abs() <= e + 2.0 ** -15 * (y.abs() + e)).all())


def reference(d_out, x, wg, wu, gates, kind):
    """The gradients at these gates, and the bounds on them."""
    r, t = ref.ROUND[x.dtype], tiny(x.dtype)
    F = wg.shape[0]
    d, x6, wg6, wu6 = (v.double() for v in (d_out, x, wg, wu))
    g, u = unpack(gates, F).double().unbind(1)
    a, slope, z = act(g, kind)
    dg, du = d * u * slope, d * a
    f = fuzz(g, z)
    eg = (d * u).abs() * 4 * f
    eg = eg + r * (dg.abs() + eg) + t
    eu = du.abs() * f
    eu = eu + r * (du.abs() + eu) + t
    dx, ex = summed(torch.cat([dg, du], 1), torch.cat([wg6, wu6]))
    ex = ex + eg @ wg6.abs() + eu @ wu6.abs()
    dwg, ewg = summed(dg.T, x6)
    dwu, ewu = summed(du.T, x6)
    ewg, ewu = ewg + eg.T @ x6.abs(), ewu + eu.T @ x6.abs()
    return [(y, (1 + r) * e + r * y.abs() + t) for y, e in ((dx, ex), (dwg, ewg), (dwu, ewu))]


def check_backward(got, want, dt):
    for y, (w, tol) in zip(got, want):
        off = y.double() - w
        assert bool((off.abs() <= tol).all())
        if w.numel() >= 64:
            floor = tiny(dt) * w.numel() ** 0.5
            assert float(off.norm()) <= ref.ROUND[dt] * float(w.norm()) + floor


# rows, dim, inner: few tokens and many, one tile and several, whole words and odd widths
SHAPES = [(1, 64, 8), (1, 1, 1), (1, 2048, 96), (3, 517, 1001), (8, 96, 40), (9, 40, 24), (16, 200, 130), (16, 2051, 17),
          (17, 64, 128), (17, 65, 1), (100, 1, 3), (129, 72, 136), (256, 64, 128), (257, 520, 264), (300, 1000, 700),
          (1001, 517, 1531), (513, 128, 8), (40, 8, 520), (2049, 192, 1288), (700, 12, 600), (90, 20, 4000), (32, 257, 300),
          (33, 2048, 136), (64, 1536, 1001), (200, 4100, 72), (260, 1030, 515)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_matches_the_formula(shape, dt):
    import gated_delta_rule_gate_gb300 as gdn
    x, wg, wu, _ = draw(*shape, dt, seed=sum(shape))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, gates = gdn.gdn_glu(x, wg, wu, want_gates=True, error_word=err)
    check_forward(out, gates, x, wg, wu, "silu")
    assert torch.equal(gdn.gdn_glu(x, wg, wu), out) and int(err) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("T", [5, 300])
def test_activations(T, kind):
    """Gates from the functions' middle to their tails."""
    import gated_delta_rule_gate_gb300 as gdn
    for dt in ("f16", "bf16"):
        for spread in (0.3, 6.0):
            x, wg, wu, d = draw(T, 136, 200, dt, seed=T, spread=spread)
            out, gates = gdn.gdn_glu(x, wg, wu, activation=kind, want_gates=True)
            check_forward(out, gates, x, wg, wu, kind)
            got = gdn.gdn_glu_backward(d, x, wg, wu, gates, activation=kind)
            check_backward(got, reference(d, x, wg, wu, gates, kind), x.dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward_matches_the_formula(shape, dt):
    import gated_delta_rule_gate_gb300 as gdn
    x, wg, wu, d = draw(*shape, dt, seed=sum(shape) + 1)
    _, gates = gdn.gdn_glu(x, wg, wu, want_gates=True)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gdn.gdn_glu_backward(d, x, wg, wu, gates, error_word=err)
    check_backward(got, reference(d, x, wg, wu, gates, "silu"), x.dtype)
    again = gdn.gdn_glu_backward(d, x, wg, wu, gates)
    assert all(torch.equal(a, b) for a, b in zip(got, again)) and int(err) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(3000, 136, 2000), (5000, 264, 1000), (20000, 72, 200)])
def test_more_tiles_than_the_device_holds(shape):
    """Each pair of blocks takes several tiles, through both accumulators, and long sums over tokens."""
    import gated_delta_rule_gate_gb300 as gdn
    x, wg, wu, d = draw(*shape, "bf16", seed=7)
    out, gates = gdn.gdn_glu(x, wg, wu, want_gates=True)
    check_forward(out, gates, x, wg, wu, "silu")
    check_backward(gdn.gdn_glu_backward(d, x, wg, wu, gates), reference(d, x, wg, wu, gates, "silu"), x.dtype)


@pytest.mark.gpu
def test_gradient_against_differences():
    """The change of sum(d_out out) along a direction, in 64 bits by a central difference."""
    import gated_delta_rule_gate_gb300 as gdn
    x, wg, wu, d = draw(70, 48, 56, "f16", seed=3)
    for kind in ("silu", "gelu", "gelu_tanh", "sigmoid"):
        _, gates = gdn.gdn_glu(x, wg, wu, activation=kind, want_gates=True)
        got = gdn.gdn_glu_backward(d, x, wg, wu, gates, activation=kind)
        bounds = reference(d, x, wg, wu, gates, kind)
        gen = torch.Generator().manual_seed(5)
        at = [t.double() for t in (x, wg, wu)]
        loss = lambda x, wg, wu: (d.double() * act(x @ wg.T, kind)[0] * (x @ wu.T)).sum()
        for i in range(3):
            v = torch.randn(at[i].shape, generator=gen, dtype=torch.double).cuda()
            h = 1e-4
            move = lambda s: [t + s * h * v if j == i else t for j, t in enumerate(at)]
            slope = (loss(*move(1)) - loss(*move(-1))) / (2 * h)
            # the kept gates are 2^-15 off, which moves a gradient by less than its operands'
            # roundings (2^-11) do; the difference itself is good to h^2
            tol = 2 * float((bounds[i][1] * v.abs()).sum()) + 1e-5 * float(slope.abs())
            assert abs(float((got[i].double() * v).sum() - slope)) <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("T", [7, 150])
def test_columns_of_wider_tensors(T):
    """Rows that lie in wider ones, whole words apart and not; what is beside them is left alone."""
    import gated_delta_rule_gate_gb300 as gdn
    for off, wide in ((8, 24), (3, 10), (0, 1)):
        D, F = 88, 136
        x, wg, wu, d = draw(T, D, F, "bf16", seed=off)
        inside = lambda t, n: torch.full((T, n + wide), 9.0, dtype=t.dtype, device="cuda")
        xw, dw, ow, dxw = inside(x, D), inside(x, F), inside(x, F), inside(x, D)
        xw[:, off:off + D], dw[:, off:off + F] = x, d
        out, gates = gdn.gdn_glu(x, wg, wu, want_gates=True)
        o, gates2 = gdn.gdn_glu(xw[:, off:off + D], wg, wu, out=ow[:, off:off + F], want_gates=True)
        assert torch.equal(o, out) and torch.equal(unpack(gates, F), unpack(gates2, F)) and o.data_ptr() == ow[:, off:off + F].data_ptr()
        want = gdn.gdn_glu_backward(d, x, wg, wu, gates)
        got = gdn.gdn_glu_backward(dw[:, off:off + F], xw[:, off:off + D], wg, wu, gates, dx=dxw[:, off:off + D])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for t, n in ((ow, F), (dxw, D)):
            assert bool((t[:, :off] == 9).all()) and bool((t[:, off + n:] == 9).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [7, 150])
def test_rows_that_end_inside_a_word(T):
    """Widths that are no multiple of 8 in rows that are whole words apart: what is behind a row
    in its last word (NaN) has no say, and is left alone."""
    import gated_delta_rule_gate_gb300 as gdn
    for D, F in ((85, 131), (1, 7), (62, 260)):
        x, wg, wu, d = draw(T, D, F, "f16", seed=D)
        nan = lambda n: torch.full((T, -(-n // 8) * 8 + 8), float("nan"), dtype=x.dtype, device="cuda")
        xw, dw, ow, dxw = nan(D), nan(F), nan(F), nan(D)
        xw[:, :D], dw[:, :F] = x, d
        out, gates = gdn.gdn_glu(x, wg, wu, want_gates=True)
        o, gates2 = gdn.gdn_glu(xw[:, :D], wg, wu, out=ow[:, :F], want_gates=True)
        assert torch.equal(o, out) and torch.equal(unpack(gates, F), unpack(gates2, F))
        want = gdn.gdn_glu_backward(d, x, wg, wu, gates)
        got = gdn.gdn_glu_backward(dw[:, :F], xw[:, :D], wg, wu, gates, dx=dxw[:, :D])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert bool(ow[:, F:].isnan().all()) and bool(dxw[:, D:].isnan().all())


@pytest.mark.gpu
def test_weights_in_one_tensor_and_at_odd_addresses():
    import gated_delta_rule_gate_gb300 as gdn
    for T in (4, 60):
        for D, F in ((64, 40), (63, 41)):
            x, wg, wu, d = draw(T, D, F, "f16", seed=D)
            flat = torch.zeros(2 * F * D + 1, dtype=x.dtype, device="cuda")
            for at in (0, 1):
                w = flat[at:at + 2 * F * D].view(2 * F, D)
                w.copy_(torch.cat([wg, wu]))
                out, gates = gdn.gdn_glu(x, w[:F], w[F:], want_gates=True)
                check_forward(out, gates, x, wg, wu, "silu")
                dw = torch.zeros_like(flat)[at:at + 2 * F * D].view(2 * F, D)
                b = gdn.gdn_glu_backward(d, x, w[:F], w[F:], gates, d_w_gate=dw[:F], d_w_up=dw[F:])
                check_backward((b.dx, dw[:F], dw[F:]), reference(d, x, wg, wu, gates, "silu"), x.dtype)


@pytest.mark.gpu
def test_leading_dimensions_and_wanted_parts():
    import gated_delta_rule_gate_gb300 as gdn
    x, wg, wu, d = draw(60, 72, 80, "bf16", seed=9)
    out, gates = gdn.gdn_glu(x.view(3, 20, 72), wg, wu, want_gates=True)
    assert out.shape == (3, 20, 80) and gates.shape == (3, 20, 768)
    flat = gdn.gdn_glu_backward(d, x, wg, wu, gates.view(60, 768))
    b = gdn.gdn_glu_backward(d.view(3, 20, 80), x.view(3, 20, 72), wg, wu, gates)
    assert b.dx.shape == (3, 20, 72) and torch.equal(b.dx.view(60, 72), flat.dx)
    one = gdn.gdn_glu(x[0], wg, wu)
    assert one.shape == (80,)
    check_forward(one[None], None, x[:1], wg, wu, "silu")
    only = gdn.gdn_glu_backward(d, x, wg, wu, gates.view(60, 768), want_d_weights=False)
    assert only.d_w_gate is None and only.d_w_up is None and torch.equal(only.dx, flat.dx)
    only = gdn.gdn_glu_backward(d, x, wg, wu, gates.view(60, 768), want_dx=False)
    assert only.dx is None and torch.equal(only.d_w_gate, flat.d_w_gate) and torch.equal(only.d_w_up, flat.d_w_up)


@pytest.mark.gpu
def test_no_tokens():
    import gated_delta_rule_gate_gb300 as gdn
    x, wg, wu, d = draw(0, 24, 16, "f16")
    out, gates = gdn.gdn_glu(x, wg, wu, want_gates=True)
    assert out.shape == (0, 16) and gates.shape == (0, 384)
    dw = [torch.full_like(wg, 5.0) for _ in range(2)]
    b = gdn.gdn_glu_backward(d, x, wg, wu, gates, d_w_gate=dw[0], d_w_up=dw[1])
    assert b.dx.shape == (0, 24) and not bool(dw[0].any()) and not bool(dw[1].any())
    assert gdn.gdn_glu_backward(d, x, wg, wu, gates, want_d_weights=False).dx.shape == (0, 24)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [6, 200])
def test_a_token_that_is_not_finite_stays_by_itself(T):
    """In an odd width too, where rows are copied beside one another."""
    import gated_delta_rule_gate_gb300 as gdn
    for D in (72, 73):
        x, wg, wu, d = draw(T, D, 90, "bf16", seed=4)
        want = gdn.gdn_glu(x, wg, wu)
        x[3] = float("nan")
        got, gates = gdn.gdn_glu(x, wg, wu, want_gates=True)
        rest = torch.arange(T, device="cuda") != 3
        assert bool(got[3].isnan().all()) and torch.equal(got[rest], want[rest])
        dx = gdn.gdn_glu_backward(d, x, wg, wu, gates, want_d_weights=False).dx
        assert bool(dx[3].isnan().all()) and bool(dx[rest].isfinite().all())


@pytest.mark.gpu
def test_same_bits_on_any_stream_and_from_a_graph():
    import gated_delta_rule_gate_gb300 as gdn
    x, wg, wu, d = draw(700, 264, 333, "bf16", seed=2)
    few = x[:3].clone()
    torch.cuda.synchronize()

    def all_of(**kw):
        out, gates = gdn.gdn_glu(x, wg, wu, want_gates=True, **kw)
        return [out, *gdn.gdn_glu_backward(d, x, wg, wu, gates, **kw), gdn.gdn_glu(few, wg, wu, **kw)]

    want = all_of()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = all_of(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 2048, 200), (30, 520, 77), (64, 2048, 136), (90, 63, 41)])
def test_every_path_from_a_graph(shape):
    """Few tokens, shares over stretches of K, copied operands: replayed on new inputs, and two
    graphs of the same call in turn."""
    import gated_delta_rule_gate_gb300 as gdn
    x, wg, wu, d = draw(*shape, "bf16", seed=8)

    def all_of():
        out, gates = gdn.gdn_glu(x, wg, wu, want_gates=True)
        return [out, *gdn.gdn_glu_backward(d, x, wg, wu, gates)]

    all_of()
    torch.cuda.synchronize()
    graphs, results = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            results.append(all_of())
    for turn in range(3):
        x.mul_(-0.5), wg.mul_(1.25), d.add_(0.125)
        want = all_of()
        for graph, got in zip(graphs, results):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_largest_values():
    """fp16 results beyond its range are infinite, gates beyond it are kept as they are."""
    import gated_delta_rule_gate_gb300 as gdn
    for T in (4, 50):
        x = torch.full((T, 64), 60.0, dtype=torch.float16, device="cuda")
        w = torch.full((24, 64), 60.0, dtype=torch.float16, device="cuda")
        out, gates = gdn.gdn_glu(x, w, w, want_gates=True)
        assert bool(out.isinf().all()) and bool((unpack(gates, 24) == 230400.0).all())
        d = torch.full((T, 24), 2.0 ** -14, dtype=torch.float16, device="cuda")
        b = gdn.gdn_glu_backward(d, x, w, w, gates)
        # d_g = d_u = 2^-14 230400 = 14.0625, an fp16 number; the sums are exact in fp32
        rounded = lambda v: float(torch.tensor(v, dtype=torch.float32).half())
        assert bool((b.dx == rounded(2 * 24 * 60 * 14.0625)).all())
        assert bool((b.d_w_gate == rounded(T * 60 * 14.0625)).all()) and torch.equal(b.d_w_gate, b.d_w_up)


@pytest.mark.gpu
def test_two_calls_at_once():
    """On two streams, each with buffers of its own."""
    import gated_delta_rule_gate_gb300 as gdn
    sets = [draw(1500, 136, 333, "f16", seed=s) for s in (1, 2)]
    want = []
    for x, wg, wu, d in sets:
        out, gates = gdn.gdn_glu(x, wg, wu, want_gates=True)
        want.append([out, *gdn.gdn_glu_backward(d, x, wg, wu, gates)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        got = []
        for (x, wg, wu, d), s in zip(sets, streams):
            out, gates = gdn.gdn_glu(x, wg, wu, want_gates=True, stream=s)
            got.append([out, gates, *gdn.gdn_glu_backward(d, x, wg, wu, gates, stream=s)])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip([a[0], *a[2:]], b))


@pytest.mark.gpu
def test_given_workspace():
    import gated_delta_rule_gate_gb300 as gdn
    x, wg, wu, d = draw(50, 63, 41, "f16", seed=6)
    out, gates = gdn.gdn_glu(x, wg, wu, want_gates=True)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    assert torch.equal(gdn.gdn_glu(x, wg, wu, workspace=ws), out)
    want = gdn.gdn_glu_backward(d, x, wg, wu, gates)
    got = gdn.gdn_glu_backward(d, x, wg, wu, gates, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(gdn.GdnError, match="workspace needs"):
        gdn.gdn_glu(x, wg, wu, workspace=small)
    with pytest.raises(gdn.GdnError, match="workspace needs"):
        gdn.gdn_glu_backward(d, x, wg, wu, gates, workspace=small)
    with pytest.raises(gdn.GdnError, match="16-bit"):
        gdn.gdn_glu(x.float(), wg.float(), wu.float())


# ---------------------------------------------------------------- refusals (no GPU)
def _forward(**over):
    a = N.GdnGluArgs()
    a.rows, a.dim, a.inner, a.dtype = 40, 24, 16, N.DTYPE_BF16
    for f in ("x", "w_gate", "w_up", "out"):
        setattr(a, f, FAKE)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def _backward(**over):
    a = N.GdnGluGradArgs()
    a.rows, a.dim, a.inner, a.dtype = 20, 24, 16, N.DTYPE_F16
    for f in ("x", "w_gate", "w_up", "d_out", "gates", "dx", "d_w_gate"):
        setattr(a, f, FAKE)
    a.d_w_up = 2 * FAKE
    for k, v in over.items():
        setattr(a, k, v)
    return a


COMMON = [
    (dict(rows=-1), N.GDN_ERR_INVALID, "rows"),
    (dict(rows=(1 << 31) - 511), N.GDN_ERR_UNSUPPORTED, "rows"),
    (dict(dim=0), N.GDN_ERR_INVALID, "dim"),
    (dict(inner=0), N.GDN_ERR_INVALID, "inner"),
    (dict(inner=(1 << 20) + 1), N.GDN_ERR_UNSUPPORTED, "inner"),
    (dict(dtype=N.DTYPE_F32), N.GDN_ERR_UNSUPPORTED, "float32"),
    (dict(dtype=N.DTYPE_E4M3), N.GDN_ERR_INVALID, "dtype"),
    (dict(activation=5), N.GDN_ERR_INVALID, "activation"),
    (dict(x_stride=23), N.GDN_ERR_INVALID, "x_stride"),
    (dict(x=FAKE + 1), N.GDN_ERR_INVALID, "aligned"),
    (dict(gates=FAKE + 8), N.GDN_ERR_INVALID, "gates"),
    (dict(error_word=FAKE + 2), N.GDN_ERR_INVALID, "aligned"),
    (dict(w_up=None), N.GDN_ERR_INVALID, "w_up"),
]


@pytest.mark.parametrize("over,status,msg", COMMON + [
    (dict(out_stride=15), N.GDN_ERR_INVALID, "out_stride"),
    (dict(out=None), N.GDN_ERR_INVALID, "out"),
    (dict(dim=23), N.GDN_ERR_WORKSPACE, "workspace"),
])
def test_forward_refuses(over, status, msg):
    a, lib = _forward(**over), N.load()
    need = lib.gdn_glu_workspace_size(ctypes.byref(a))
    assert (need == ctypes.c_size_t(-1).value) == (status != N.GDN_ERR_WORKSPACE)
    assert lib.gdn_glu(ctypes.byref(a), None, 0, None) == status
    assert msg.lower() in N.last_error_message().lower()
    assert lib.gdn_glu(None, None, 0, None) == N.GDN_ERR_INVALID


@pytest.mark.parametrize("over,status,msg", COMMON + [
    (dict(d_out_stride=15), N.GDN_ERR_INVALID, "d_out_stride"),
    (dict(dx_stride=8), N.GDN_ERR_INVALID, "dx_stride"),
    (dict(d_out=None), N.GDN_ERR_INVALID, "d_out"),
    (dict(x=None), N.GDN_ERR_INVALID, "x is"),
    (dict(d_w_up=None), N.GDN_ERR_INVALID, "go together"),
    (dict(d_w_up=FAKE), N.GDN_ERR_INVALID, "one tensor"),
    (dict(dx=None, d_w_gate=None, d_w_up=None), N.GDN_ERR_INVALID, "required"),
    (dict(), N.GDN_ERR_WORKSPACE, "workspace"),
])
def test_backward_refuses(over, status, msg):
    a, lib = _backward(**over), N.load()
    need = lib.gdn_glu_backward_workspace_size(ctypes.byref(a))
    assert (need == ctypes.c_size_t(-1).value) == (status != N.GDN_ERR_WORKSPACE)
    assert lib.gdn_glu_backward(ctypes.byref(a), None, 0, None) == status
    assert msg.lower() in N.last_error_message().lower()
    assert lib.gdn_glu_backward(None, None, 0, None) == N.GDN_ERR_INVALID


def test_whole_words_need_no_workspace():
    lib = N.load()
    assert lib.gdn_glu_workspace_size(ctypes.byref(_forward())) == 0
    assert lib.gdn_glu_workspace_size(ctypes.byref(_forward(x=FAKE + 2))) > 0
    assert lib.gdn_glu_workspace_size(ctypes.byref(_forward(x=FAKE + 2, rows=3))) == 0


def test_binding_refuses():
    import gated_delta_rule_gate_gb300 as gdn
    from layer_standins import Standin
    h = torch.float16
    S = lambda *s, **kw: Standin(s, **{"dtype": h, **kw})
    x, w, d, gates = S(20, 24), S(16, 24), S(20, 16), Standin((20, 384), dtype=torch.uint8)
    glu, back = gdn.gdn_glu, gdn.gdn_glu_backward
    for call, exc, msg in [
        (lambda: glu(x, w), TypeError, "w_up"),
        (lambda: glu(x, w, None), TypeError, "w_up"),
        (lambda: glu(x, S(16, 25), w), ValueError, "w_gate must be"),
        (lambda: glu(x, w, S(17, 24)), ValueError, "w_up must be"),
        (lambda: glu(x, S(24), w), ValueError, "w_gate must be"),
        (lambda: glu(x, w, S(16, 24, dtype=torch.bfloat16)), TypeError, "w_up"),
        (lambda: glu(x, w, w, activation="tanh"), ValueError, "activation"),
        (lambda: glu(x, w, w, activation=3), ValueError, "activation"),
        (lambda: glu(x, w, w, out=S(20, 17)), ValueError, "out must be"),
        (lambda: glu(x, w, w, out=Standin((20, 16), (0, 1), dtype=h)), ValueError, "overlap"),
        (lambda: glu(Standin((20, 24), (1, 20), dtype=h), w, w), ValueError, "contiguous"),
        (lambda: glu(x, Standin((16, 24), (1, 16), dtype=h), w), ValueError, "contiguous"),
        (lambda: glu(x, S(16, 24, device="cuda:1"), w), ValueError, "cuda:1"),
        (lambda: glu(x, w, w, workspace=torch.zeros(4)), ValueError, "cpu"),
        (lambda: glu(torch.zeros(20, 24, dtype=h), torch.zeros(16, 24, dtype=h), torch.zeros(16, 24, dtype=h)),
         ValueError, "cpu"),
        (lambda: glu(S(20, 24, dtype=torch.int32), w, w), TypeError, "dtype"),
        (lambda: back(S(20, 17), x, w, w, gates), ValueError, "d_out must be"),
        (lambda: back(d, x, w, w, S(20, 16)), ValueError, "gates must be"),
        (lambda: back(d, x, w, w, S(20, 384, dtype=torch.float32)), TypeError, "gates"),
        (lambda: back(d, x, w, w, gates, dx=S(20, 16)), ValueError, "dx must be"),
        (lambda: back(d, x, w, w, gates, want_dx=False, dx=x), ValueError, "want_dx"),
        (lambda: back(d, x, w, w, gates, want_d_weights=False, d_w_up=w), ValueError, "want_d_weights"),
        (lambda: back(d, x, w, w, gates, d_w_gate=S(24, 16)), ValueError, "d_w_gate must be"),
        (lambda: back(d, x, w, w, Standin((20, 384), dtype=torch.uint8, device="cuda:1")), ValueError, "cuda:1"),
    ]:
        with pytest.raises(exc, match=msg):
            call()
