"""gdn_rmsnorm and gdn_rmsnorm_backward against their formulas in 64 bits and
against differences, and their refusals.

Tolerances.  A row's sum of D squares in fp32 partial sums is off by at most
(log2(1024) + values a thread) * 2^-24 of it, far under 64 * 2^-24 = 4e-6, halved by
the root; the products add a few 2^-24: TOL = 1e-5 relative to the largest value,
plus the rounding of a 16-bit output.  E4M3 keeps 3 bits of mantissa: a value of a
row is off by at most 2^-4 of itself, or half a step (2^-10) of the smallest ones, and
by TOL before the rounding.  d_weight sums `rows` terms in fp32: rows * 2^-24 of the
sum of their sizes at most, and TOL of each term.
"""
import ctypes
import math

import pytest
import torch

import layer_reference as ref
from gated_delta_rule_gate_gb300 import _native as N

TOL = 1e-5
FAKE = 0x100000
E4M3 = torch.float8_e4m3fn


def draw(seed, n, D, act, residual, weight="same", std=1.0):
    gen = torch.Generator().manual_seed(seed)
    dt = ref.DT[act]
    x = (torch.randn(n, D, generator=gen) * std).to(dt)
    res = None if residual is None else torch.randn(n, D, generator=gen).to(dt if residual == "same" else torch.float32)
    w = (1 + 0.3 * torch.randn(D, generator=gen)).to(dt if weight == "same" else torch.float32)
    return x, res, w


def formula(x, res, w, eps):
    r = x.double() if res is None else x.double() + res.double()
    rstd = 1 / torch.sqrt((r * r).mean(1) + eps)
    return r, rstd, r * rstd[:, None] * w.double()


def check_e4m3(out, scales, y, group):
    n, D = y.shape
    out, scales = out.float().double().cpu(), scales.double().cpu()
    g = group or D
    groups = y.split(g, dim=1)
    want = torch.stack([p.abs().amax(1) for p in groups], 1) / 448
    got = scales.view(n, -1)
    assert bool(((got - want).abs() <= TOL * want + 2.0 ** -100).all())
    scale = got.repeat_interleave(g, dim=1)[:, :D]
    v = out * scale
    assert bool(((v - y).abs() <= y.abs() * (2.0 ** -4 + TOL) + scale * 2.0 ** -10 + TOL * y.abs().amax()).all())
    # the largest value of each group stands near the type's largest
    top = torch.stack([p.abs().amax(1) for p in out.split(g, dim=1)], 1)
    assert bool(((top >= 416) | (want <= 2.0 ** -100)).all()) and bool((top <= 448).all())


SHAPES = [(1, 1), (3, 7), (2, 128), (5, 129), (4, 130), (1, 2048), (7, 517), (3, 1531), (2, 4096), (2, 5000), (3, 8192),
          (2, 8200), (2, 16384), (1, 20001)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,D", SHAPES)
@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
def test_matches_the_formula(n, D, act):
    import gated_delta_rule_gate_gb300 as g
    for k, residual in enumerate([None, "same", "f32"]):
        x, res, w = draw(D + k, n, D, act, residual, weight="f32" if k == 1 else "same")
        r, rstd, y = formula(x, res, w, 1e-5)
        c = lambda t: None if t is None else t.cuda()
        got = g.gdn_rmsnorm(c(x), c(w), residual=c(res), eps=1e-5, want_rstd=True)
        assert got.out.dtype == x.dtype and ref.rel(got.out, y) <= TOL + ref.ROUND[x.dtype]
        assert got.residual is None if res is None else ref.rel(got.residual, r) <= TOL + ref.ROUND[res.dtype]
        assert ref.rel(got.rstd, rstd) <= TOL and got.scales is None
        for group in (0, 128):
            q = g.gdn_rmsnorm(c(x), c(w), residual=c(res), eps=1e-5, out_dtype=E4M3, group=group)
            assert q.out.dtype == E4M3 and q.scales.shape == ((n,) if not group else (n, -(-D // 128)))
            check_e4m3(q.out, q.scales, y, group)
            assert res is None or torch.equal(q.residual, got.residual)


@pytest.mark.gpu
def test_residual_in_place_strides_and_leading_dimensions():
    import gated_delta_rule_gate_gb300 as g
    for D in (256, 130, 20001):
        x, res, w = (t.cuda() for t in draw(1, 12, D, "f16", "f32"))
        want = g.gdn_rmsnorm(x, w, residual=res)
        stream = res.clone()
        got = g.gdn_rmsnorm(x.view(3, 4, D), w, residual=stream.view(3, 4, D), residual_out=stream.view(3, 4, D))
        assert got.out.shape == (3, 4, D) and torch.equal(got.out.view(12, D), want.out)
        assert torch.equal(stream, want.residual)
        for off in (0, 3, 8):
            wide = torch.zeros(12, D + 24, dtype=torch.half, device="cuda")
            wide[:, off:off + D] = x
            assert torch.equal(g.gdn_rmsnorm(wide[:, off:off + D], w, residual=res).out, want.out)


@pytest.mark.gpu
def test_rows_of_zeros_infinities_and_nan():
    """Zeros give zeros and a positive scale; a row that is not finite spoils no other."""
    import gated_delta_rule_gate_gb300 as g
    for D in (512, 517):
        x = torch.randn(5, D, generator=torch.Generator().manual_seed(2))
        x[1] = 0
        x[2, 3] = math.inf
        x[3, 4] = math.nan
        x[4, :300] = 0  # whole groups of zeros
        w = torch.ones(D)
        ok = [0, 1, 4]
        _, _, y = formula(x[ok], None, w, 1e-6)
        plain = g.gdn_rmsnorm(x.cuda(), w.cuda()).out
        assert ref.rel(plain[ok], y) <= TOL and bool(torch.isnan(plain[3]).all())
        for group in (0, 128):
            q = g.gdn_rmsnorm(x.cuda(), w.cuda(), out_dtype=E4M3, group=group)
            check_e4m3(q.out[ok], q.scales[ok], y, group)
            assert bool((q.scales[ok] > 0).all()) and bool(torch.isnan(q.out[3].float()).all())


@pytest.mark.gpu
def test_large_values_do_not_overflow():
    """Sums of squares of half the largest fp16 values, in fp32."""
    import gated_delta_rule_gate_gb300 as g
    x, _, w = draw(3, 2, 4096, "f16", None, std=16000.0)
    x = x.clamp(-60000, 60000)
    _, _, y = formula(x, None, w, 1e-6)
    assert ref.rel(g.gdn_rmsnorm(x.cuda(), w.cuda()).out, y) <= TOL + ref.ROUND[torch.float16]


def gradient(d_out, r, w, rstd, d_res):
    d, r, w, rstd = d_out.double(), r.double(), w.double(), rstd.double()[:, None]
    xhat = r * rstd
    m = (d * w * xhat).mean(1, keepdim=True)
    dx = rstd * (d * w - xhat * m)
    if d_res is not None:
        dx = dx + d_res.double()
    return dx, (d * xhat).sum(0), (d * xhat).abs().sum(0)


@pytest.mark.gpu
@pytest.mark.parametrize("n,D", SHAPES + [(700, 64), (1500, 33), (650, 8200)])
@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
def test_gradient_matches_the_formula(n, D, act):
    import gated_delta_rule_gate_gb300 as g
    gen = torch.Generator().manual_seed(n)
    for k, residual in enumerate([None, "same", "f32"]):
        x, res, w = draw(D + k, n, D, act, residual, weight="f32" if k == 2 else "same")
        r = x if res is None else (x.float() + res.float()).to(res.dtype)
        rstd = formula(r, None, w, 1e-5)[1].float()
        d_out = torch.randn(n, D, generator=gen).to(x.dtype)
        d_res = torch.randn(n, D, generator=gen).to(r.dtype) if k else None
        dx, dw, size = gradient(d_out, r, w, rstd, d_res)
        c = lambda t: None if t is None else t.cuda()
        got = g.gdn_rmsnorm_backward(c(d_out), c(r), c(w), c(rstd), d_residual=c(d_res))
        assert got.dx.dtype == r.dtype and ref.rel(got.dx, dx) <= TOL + ref.ROUND[r.dtype]
        assert bool(((got.dweight.double().cpu() - dw).abs() <= (n * 2.0 ** -24 + TOL) * size + 1e-30).all())
        if d_res is not None:  # in place
            acc = c(d_res)
            again = g.gdn_rmsnorm_backward(c(d_out), c(r), c(w), c(rstd), d_residual=acc, dx=acc)
            assert torch.equal(again.dx, got.dx) and torch.equal(again.dweight, got.dweight)


@pytest.mark.gpu
def test_gradient_against_differences():
    import gated_delta_rule_gate_gb300 as g
    x, res, w = draw(9, 20, 70, "f32", "f32")
    gen = torch.Generator().manual_seed(4)
    d_out, d_res = torch.randn(20, 70, generator=gen), torch.randn(20, 70, generator=gen)
    f = g.gdn_rmsnorm(x.cuda(), w.cuda(), residual=res.cuda(), want_rstd=True)
    b = g.gdn_rmsnorm_backward(d_out.cuda(), f.residual, w.cuda(), f.rstd, d_residual=d_res.cuda())

    def loss(x, res, w):
        r, _, y = formula(x, res, w, 1e-6)
        return float((y * d_out.double()).sum() + (r * d_res.double()).sum())

    for name, grad in (("x", b.dx), ("res", b.dx), ("w", b.dweight)):
        at = {"x": x.double(), "res": res.double(), "w": w.double()}
        way = torch.randn(at[name].shape, generator=gen).double()
        eps = 1e-5
        diff = (loss(**dict(at, **{name: at[name] + eps * way})) - loss(**dict(at, **{name: at[name] - eps * way}))) / (2 * eps)
        terms = grad.double().cpu() * way
        assert abs(float(terms.sum()) - diff) <= 3e-5 * float(terms.abs().sum()) + 1e-6, name


@pytest.mark.gpu
def test_same_bits_on_any_stream_and_no_rows():
    import gated_delta_rule_gate_gb300 as g
    x, res, w = (t.cuda() for t in draw(5, 3000, 520, "bf16", "f32"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    first = None
    for stream in (None, side, None):
        f = g.gdn_rmsnorm(x, w, residual=res, want_rstd=True, stream=stream)
        b = g.gdn_rmsnorm_backward(x, f.residual, w, f.rstd, stream=stream)
        torch.cuda.synchronize()
        first = first or (f, b)
        assert all(torch.equal(p, q) for p, q in zip((f.out, f.residual, f.rstd) + b,
                                                     (first[0].out, first[0].residual, first[0].rstd) + first[1]))
    none = torch.empty(0, 64, device="cuda")
    one = torch.ones(64, device="cuda")
    assert g.gdn_rmsnorm(none, one).out.shape == (0, 64)
    b = g.gdn_rmsnorm_backward(none, none, one, none[:, 0])
    assert b.dx.shape == (0, 64) and not bool(b.dweight.any())


def _args(**over):
    a = N.GdnRmsnormArgs(4, 16, N.DTYPE_F16, N.DTYPE_F16, N.DTYPE_F16, N.DTYPE_F16, 0, 1e-6, 0, FAKE, None, FAKE, FAKE)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status,msg", [
    (dict(rows=-1), N.GDN_ERR_INVALID, "rows"),
    (dict(rows=1 << 31), N.GDN_ERR_UNSUPPORTED, "rows"),
    (dict(dim=0), N.GDN_ERR_INVALID, "dim"),
    (dict(dim=(1 << 20) + 1), N.GDN_ERR_UNSUPPORTED, "dim"),
    (dict(x_dtype=N.DTYPE_E4M3), N.GDN_ERR_INVALID, "x_dtype"),
    (dict(residual=FAKE, residual_out=FAKE, residual_dtype=N.DTYPE_BF16), N.GDN_ERR_INVALID, "residual_dtype"),
    (dict(weight_dtype=N.DTYPE_BF16), N.GDN_ERR_INVALID, "weight_dtype"),
    (dict(out_dtype=N.DTYPE_F32), N.GDN_ERR_INVALID, "out_dtype"),
    (dict(group=128), N.GDN_ERR_INVALID, "group"),
    (dict(group=64, out_dtype=N.DTYPE_E4M3, scales=FAKE), N.GDN_ERR_INVALID, "group"),
    (dict(out_dtype=N.DTYPE_E4M3), N.GDN_ERR_INVALID, "scales"),
    (dict(scales=FAKE), N.GDN_ERR_INVALID, "scales"),
    (dict(eps=-1.0), N.GDN_ERR_INVALID, "eps"),
    (dict(eps=math.nan), N.GDN_ERR_INVALID, "eps"),
    (dict(residual=FAKE), N.GDN_ERR_INVALID, "residual_out"),
    (dict(x_stride=15), N.GDN_ERR_INVALID, "x_stride"),
    (dict(weight=None), N.GDN_ERR_INVALID, "required"),
    (dict(x=FAKE + 1), N.GDN_ERR_INVALID, "aligned"),
])
def test_refuses(over, status, msg):
    assert N.load().gdn_rmsnorm(ctypes.byref(_args(**over)), None) == status
    assert msg.lower() in N.last_error_message().lower()


@pytest.mark.parametrize("over,status,msg", [
    (dict(rows=-1), N.GDN_ERR_INVALID, "rows"),
    (dict(r_dtype=N.DTYPE_BF16), N.GDN_ERR_INVALID, "r_dtype"),
    (dict(d_weight=None), N.GDN_ERR_INVALID, "d_weight"),
    (dict(rstd=None), N.GDN_ERR_INVALID, "required"),
    (dict(d_out_stride=3), N.GDN_ERR_INVALID, "d_out_stride"),
    (dict(rstd=FAKE + 2), N.GDN_ERR_INVALID, "aligned"),
    (dict(), N.GDN_ERR_WORKSPACE, "workspace"),
])
def test_gradient_refuses(over, status, msg):
    a = N.GdnRmsnormGradArgs(4, 16, N.DTYPE_F16, N.DTYPE_F16, N.DTYPE_F16, 0, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE)
    for k, v in over.items():
        setattr(a, k, v)
    lib = N.load()
    need = lib.gdn_rmsnorm_backward_workspace_size(ctypes.byref(a))
    assert (need == ctypes.c_size_t(-1).value) == (status != N.GDN_ERR_WORKSPACE)
    for ws, size in ((None, 1 << 20), (FAKE, need - 1), (FAKE + 8, 1 << 20)):
        assert lib.gdn_rmsnorm_backward(ctypes.byref(a), ws, size, None) == status
        assert msg.lower() in N.last_error_message().lower()
