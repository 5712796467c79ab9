"""gdn_grad_clip against the formula in 64 bits, and its refusals.

Tolerances.  A thread adds up at most a few thousand squares in fp32, in several
partial sums, and the rest is joined in 64 bits: the norm (its root) is held to
1e-5.  A scaled value carries the factor's error and a rounding of its type.
"""
import ctypes
import math

import pytest
import torch

import layer_reference as ref
from gated_delta_rule_gate_gb300 import _native as N

TOL = 1e-5
FAKE = 0x100000


def draw(seed, sizes, types=("f32",), std=0.1):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=gen) * std).to(ref.DT[types[i % len(types)]]).cuda() for i, n in enumerate(sizes)]


def norm_of(grads):
    return math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in grads))


def check(grads, before, norm, max_norm, eps=1e-6):
    want = norm_of(before)
    assert abs(float(norm) - want) <= TOL * want + 1e-30
    k = min(1.0, max_norm / (want + eps)) if want + eps > 0 else 1.0
    for g, b in zip(grads, before):
        y = b.double() * k
        assert bool(((g.double() - y).abs() <= (TOL + ref.ROUND[g.dtype]) * y.abs() + 2.0 ** -25).all())


LISTS = [
    ([1], ("f32",)),
    ([0, 5, 0], ("f16",)),
    ([8192, 8193, 8191, 3], ("bf16", "f32")),
    ([100000, 1, 17, 65536, 12345], ("f32", "f16", "bf16")),
    ([300 + i for i in range(33)], ("f32", "bf16")),
    ([64 + i % 7 for i in range(1100)], ("f16", "f32")),
    ([3000001], ("f32",)),
    ([12000000, 7], ("bf16",)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(LISTS)))
def test_matches_the_formula(i):
    import gated_delta_rule_gate_gb300 as g
    for factor in (0.3, 5.0):  # clipped, and left alone
        grads = draw(i, *LISTS[i])
        before = [t.clone() for t in grads]
        bound = factor * norm_of(grads)
        out = [torch.full_like(t, math.nan) for t in grads]
        norm = g.gdn_grad_clip(grads, bound, out=out)
        check(out, before, norm, bound)
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
        assert torch.equal(g.gdn_grad_clip(grads, bound), norm)
        assert all(torch.equal(a, b) for a, b in zip(grads, out))


@pytest.mark.gpu
def test_parts_of_a_buffer_and_odd_addresses():
    """Tensors that begin anywhere in one flat buffer; what lies between is left alone."""
    import gated_delta_rule_gate_gb300 as g
    for dt in ("f32", "f16"):
        flat = draw(3, [70000], (dt,))[0]
        before = flat.clone()
        parts = [flat[1:9], flat[9:20001], flat[20003:20003], flat[30007:60000]]
        old = [p.clone() for p in parts]
        check(parts, old, g.gdn_grad_clip(parts, 1.0), 1.0)
        for a, b in ((0, 1), (20001, 30007), (60000, 70000)):
            assert torch.equal(flat[a:b], before[a:b])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradient_and_result_at_any_address(dt):
    """Every pair of offsets from a 16-byte address, shorter than a word and longer."""
    import gated_delta_rule_gate_gb300 as g
    for n in (1, 5, 8, 15, 9001):
        for a in range(8):
            for b in (0, a, (a + 3) % 8):
                flat = draw(n + a, [n + 16], (dt,))[0]
                out = torch.full_like(flat, 7.0)
                bound = 0.3 * norm_of([flat[a:a + n]])
                norm = g.gdn_grad_clip([flat[a:a + n]], bound, out=[out[b:b + n]])
                check([out[b:b + n]], [flat[a:a + n]], norm, bound)
                assert bool((out[:b] == 7.0).all()) and bool((out[b + n:] == 7.0).all())


@pytest.mark.gpu
def test_norms_that_are_zero_or_not_finite():
    import gated_delta_rule_gate_gb300 as g
    zero = [torch.zeros(100, device="cuda")]
    assert float(g.gdn_grad_clip(zero, 0.0, eps=0.0)) == 0 and not bool(zero[0].any())
    assert float(g.gdn_grad_clip([], 1.0)) == 0
    for bad in (math.inf, math.nan):
        grads = draw(5, [1000, 50])
        grads[1][7] = bad
        before = [t.clone() for t in grads]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        norm = float(g.gdn_grad_clip(grads, 0.1, error_word=err))
        assert (math.isnan(norm) if math.isnan(bad) else norm == math.inf) and int(err) == N.DEVERR_NONFINITE
        assert all(torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0)) for a, b in zip(grads, before))
    grads = draw(6, [1000])
    g.gdn_grad_clip(grads, 0.0)  # a bound of zero
    assert not bool(grads[0].any())


@pytest.mark.gpu
def test_same_bits_on_any_stream():
    import gated_delta_rule_gate_gb300 as g
    grads = draw(8, [500000, 3, 70001], ("bf16", "f32"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    first = None
    for stream in (None, side, None):
        out = [torch.empty_like(t) for t in grads]
        norm = g.gdn_grad_clip(grads, 1.0, out=out, stream=stream)
        torch.cuda.synchronize()
        first = first or (norm, out)
        assert torch.equal(norm, first[0]) and all(torch.equal(a, b) for a, b in zip(out, first[1]))


def _args(count=2, grads=(FAKE, FAKE), outs=None, sizes=(4, 4), dtypes=(0, 1), max_norm=1.0, eps=1e-6, **over):
    vp = ctypes.c_void_p * len(grads)
    a = N.GdnGradClipArgs(count, max_norm, eps, vp(*grads), None if outs is None else vp(*outs),
                          (ctypes.c_int64 * len(sizes))(*sizes), (ctypes.c_int32 * len(dtypes))(*dtypes))
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status,msg", [
    (dict(count=-1), N.GDN_ERR_INVALID, "count"),
    (dict(max_norm=-1.0), N.GDN_ERR_INVALID, "max_norm"),
    (dict(max_norm=math.nan), N.GDN_ERR_INVALID, "max_norm"),
    (dict(eps=-1.0), N.GDN_ERR_INVALID, "eps"),
    (dict(dtypes=(0, 3)), N.GDN_ERR_INVALID, "tensor 1"),
    (dict(sizes=(-1, 4)), N.GDN_ERR_INVALID, "tensor 0"),
    (dict(sizes=((1 << 42) + 1, 4)), N.GDN_ERR_UNSUPPORTED, "2^42"),
    (dict(grads=(FAKE, None)), N.GDN_ERR_INVALID, "tensor 1"),
    (dict(outs=(None, FAKE)), N.GDN_ERR_INVALID, "tensor 0"),
    (dict(grads=(FAKE + 2, FAKE)), N.GDN_ERR_INVALID, "aligned"),
    (dict(norm=FAKE + 1), N.GDN_ERR_INVALID, "aligned"),
    (dict(), N.GDN_ERR_WORKSPACE, "workspace"),
])
def test_refuses(over, status, msg):
    a = _args(**over)
    lib = N.load()
    need = lib.gdn_grad_clip_workspace_size(ctypes.byref(a))
    assert (need == ctypes.c_size_t(-1).value) == (status != N.GDN_ERR_WORKSPACE)
    assert lib.gdn_grad_clip(ctypes.byref(a), None, 0, None) == status
    assert msg.lower() in N.last_error_message().lower()
    assert lib.gdn_grad_clip(None, None, 0, None) == N.GDN_ERR_INVALID


def test_binding_refuses():
    import gated_delta_rule_gate_gb300 as g
    t = torch.zeros(4)
    with pytest.raises(ValueError, match="device"):
        g.gdn_grad_clip([t], 1.0, norm=t[:1])
