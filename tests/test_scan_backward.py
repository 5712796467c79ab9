"""gdn_scan_backward against the formula in 64 bits and against differences, and
its refusals.

Tolerances.  The states h and the handed-back gradients c are recurrences of the
kind that the forward tests hold to 1e-4 (memory of up to 200 tokens); a gradient
is a product of at most two of them with gate factors that carry a few 2^-24:
3e-4 relative to the largest value, plus the rounding of a 16-bit output.  The sums
over tokens are held to 3e-4 of the sum of their terms' sizes.
"""
import ctypes
import math

import pytest
import torch

import layer_reference as ref
from gated_delta_rule_gate_gb300 import _native as N
from test_scan import CASES, FAKE, _args, draw, lens_clamped

TOL = 3e-4


def run(p, seed, final=True, fill=math.nan, stream=None, err=None):
    """Forward and backward on the GPU; returns the gradients' inputs and results."""
    import gated_delta_rule_gate_gb300 as g
    gen = torch.Generator().manual_seed(seed)
    d_out = torch.randn(p["x"].shape, generator=gen).to(p["x"].dtype)
    D = p["x"].shape[-1]
    d_fin = torch.randn(p["nrows"], D, generator=gen) if final else None
    c = lambda t: None if t is None else t.cuda()
    i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")
    kw = dict(beta=c(p["beta"]), gate_bias=c(p["bias"]), gate_scale=c(p["scale"]),
              beta_sigmoid=p["sigmoid"] and p["beta"] is not None, input_scale=p["mode"], cu_seqlens=c(p["cu"]),
              seq_lens=i32(p["seq_lens"]), slot_ids=i32(p["slots"]), initial_state=c(p["h0"]), error_word=err,
              stream=stream)
    x, z = c(p["x"]), c(p["decay"])
    _, chunks = g.gdn_scan(x, z, want_chunk_states=True, **kw)
    full = lambda t: None if t is None else torch.full(t.shape, fill, dtype=t.dtype, device="cuda")
    got = g.gdn_scan_backward(c(d_out), x, z, chunks, d_final_state=c(d_fin), dx=full(x), d_decay=full(z),
                              d_beta=full(p["beta"]), d_initial_state=full(p["h0"]), **kw)
    return d_out, d_fin, got


def check(p, d_out, d_fin, got):
    _, _, want = ref.scan(p, (d_out, d_fin))
    D = p["x"].shape[-1]
    for name, like in (("dx", p["x"]), ("d_decay", p["decay"]), ("d_beta", p["beta"])):
        t = getattr(got, name)
        if like is None:
            assert t is None
            continue
        assert t.dtype == like.dtype and t.shape == like.shape
        assert ref.rel(t, want[name]) <= TOL + ref.ROUND[like.dtype], name
        assert bool(torch.isnan(t.float().cpu().reshape(-1, D)[torch.isnan(want[name])]).all())  # not written
    if p["bias"] is not None:
        for name, size in zip(("d_gate_bias", "d_gate_scale"), want["sum_of_sizes"]):
            err = (getattr(got, name).double().cpu() - want[name]).abs()
            assert bool((err <= TOL * size.max() + 1e-30).all()), name
    if p["h0"] is not None:
        t = got.d_initial_state
        assert ref.rel(t, want["d_initial_state"]) <= TOL
        assert bool(torch.isnan(t.cpu()[torch.isnan(want["d_initial_state"])]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_the_formula(i):
    c = CASES[i]
    p = draw(500 + i, **lens_clamped(c))
    if c.get("seq_lens"):
        p["seq_lens"] = c["seq_lens"]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(p, *run(p, i, final=i % 3 != 2, err=err))
    assert int(err) == (N.DEVERR_BAD_SLOT if None in p["rows"] else 0)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("mode", ["none", "lerp", "unit"])
@pytest.mark.parametrize("raw", [True, False])
def test_types_and_gates(act, mode, raw):
    for k, beta in enumerate([None, "plain", "sigmoid"]):
        p = draw(700 + k, 150, lengths=[200, 1, 0, 333], act=act, mode=mode, raw=raw, beta=beta,
                 gate="f32" if k == 1 else "same")
        check(p, *run(p, k))


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["none", "lerp", "unit"])
def test_against_differences(mode):
    """Directional differences of the 64-bit forward pass, input by input."""
    p = draw(41, 70, lengths=[150, 0, 1, 90], mode=mode)
    d_out, d_fin, got = run(p, 3)
    gen = torch.Generator().manual_seed(9)

    def loss(q):
        out, fin = ref.scan(q)
        return float((out * d_out.double()).sum() + (fin * d_fin.double()).sum())

    grads = {"x": got.dx, "decay": got.d_decay, "beta": got.d_beta, "bias": got.d_gate_bias,
             "scale": got.d_gate_scale, "h0": got.d_initial_state}
    for name, grad in grads.items():
        way = torch.randn(p[name].shape, generator=gen).double()
        eps = 1e-5
        base = p[name].double()
        diff = (loss(dict(p, **{name: base + eps * way})) - loss(dict(p, **{name: base - eps * way}))) / (2 * eps)
        terms = grad.double().cpu() * way
        # the gradient's own tolerance on each term; the differences are exact to about eps^2 and 1e-16 / eps
        assert abs(float(terms.sum()) - diff) <= TOL * float(terms.abs().sum()) + 1e-6, name


@pytest.mark.gpu
def test_a_request_does_not_see_its_neighbours():
    p = draw(51, 66, lengths=[70, 64, 61, 200], mode="lerp")
    d_out, d_fin, _ = run(p, 1)
    _, _, want = ref.scan(p, (d_out, d_fin))
    bad = dict(p, x=p["x"].clone(), h0=p["h0"].clone())
    bad["x"][p["spans"][1][0] + 2] = math.nan
    bad["h0"][1] = math.inf
    _, _, got = run(bad, 1)
    for b in (0, 2, 3):
        t0, t1 = p["spans"][b]
        for name in ("dx", "d_decay", "d_beta"):
            assert ref.rel(getattr(got, name)[t0:t1], want[name][t0:t1]) <= TOL
        assert ref.rel(got.d_initial_state[b], want["d_initial_state"][b]) <= TOL


@pytest.mark.gpu
def test_same_bits_on_every_run_and_any_stream():
    p = draw(61, 1100, lengths=[3000, 77, 1500], act="bf16", mode="unit")
    first = run(p, 2)[2]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side):
        again = run(p, 2, stream=stream)[2]
        torch.cuda.synchronize()
        for a, b in zip(first, again):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_allocated_gradients_of_tokens_without_a_request_are_zero():
    import gated_delta_rule_gate_gb300 as g
    x = torch.randn(40, 12, device="cuda")
    z = -torch.rand(40, 12, device="cuda")
    cu = torch.tensor([3, 10, 30], dtype=torch.int32, device="cuda")
    out, chunks = g.gdn_scan(x, z, cu_seqlens=cu, want_chunk_states=True)
    r = g.gdn_scan_backward(torch.ones_like(x), x, z, chunks, cu_seqlens=cu)
    assert not bool(r.dx[:3].any()) and not bool(r.dx[30:].any()) and bool(r.dx[3:30].all())
    assert not bool(r.d_decay[:3].any()) and not bool(r.d_decay[30:].any())
    assert r.d_beta is None and r.d_gate_bias is None and r.d_initial_state is None


def _grad_args(forward=None, **over):
    f = _args(chunk_states=FAKE, o=None, **(forward or {}))
    a = N.GdnScanGradArgs(f, 0, 0, 0, 0, FAKE, None, FAKE, FAKE)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("forward,over,msg", [
    (dict(chunk_states=None), {}, "chunk_states"),
    (dict(channels=-4), {}, "channels"),
    ({}, dict(d_o=None), "required"),
    ({}, dict(dx=None), "required"),
    ({}, dict(d_decay=None), "required"),
    (dict(beta=FAKE), {}, "d_beta is required"),
    ({}, dict(d_beta=FAKE), "without beta"),
    ({}, dict(d_gate_bias=FAKE), "raw-gate"),
    ({}, dict(dx_stride=3), "dx_stride"),
    ({}, dict(d_o=FAKE + 1), "aligned"),
    ({}, dict(d_initial_state=FAKE + 2), "aligned"),
])
def test_refuses(forward, over, msg):
    a = _grad_args()
    for k, v in forward.items():
        setattr(a.forward, k, v)
    for k, v in over.items():
        setattr(a, k, v)
    assert N.load().gdn_scan_backward(ctypes.byref(a), None) == N.GDN_ERR_INVALID
    assert msg.lower() in N.last_error_message().lower()
    assert N.load().gdn_scan_backward(None, None) == N.GDN_ERR_INVALID
