"""gdn_adamw refuses a tensor that is listed twice, in one list or in two."""
import ctypes
import itertools

import pytest

import test_adamw as adamw
from gated_delta_rule_gate_gb300 import _native as N

AT = 0x10000000
LISTS = ("params", "exp_avg", "exp_avg_sq", "exp_avg_scales", "exp_avg_sq_scales", "master")


def apart(n, reverse=False):
    """Addresses of n tensors of each list, a megabyte apart, rising or falling."""
    at = {k: [AT + (j * n + i) * (1 << 20) for i in range(n)] for j, k in enumerate(LISTS)}
    return {k: v[::-1] if reverse else v for k, v in at.items()}


def call(n, sizes, eight, at, **over):
    at = {k: v for k, v in at.items() if eight or "scales" not in k}
    a = adamw._args(n, state_dtype=N.DTYPE_E4M3 if eight else N.DTYPE_F32, sizes=sizes, param_dtypes=[1] * n,
                    grad_dtypes=[1] * n, **at, **over)
    status = N.load().gdn_adamw(ctypes.byref(a), None)
    return status, N.last_error_message()


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("n", [2, 30, 64, 65, 500])
@pytest.mark.parametrize("name", LISTS)
def test_refuses_a_tensor_twice(name, n, reverse):
    sizes = [300 + i for i in range(n)]
    at = apart(n, reverse)
    at[name][n - 1] = at[name][0]
    status, message = call(n, sizes, True, at)
    assert status == N.GDN_ERR_INVALID
    assert message == "%s[%d] is %s[0]: one tensor twice" % (name, n - 1, name)


@pytest.mark.parametrize("first,second", list(itertools.combinations(LISTS, 2)))
def test_refuses_one_tensor_for_two_parts(first, second):
    at = apart(3)
    at[second][1] = at[first][1]
    status, message = call(3, [300] * 3, True, at)
    assert status == N.GDN_ERR_INVALID
    assert message == "%s[1] is %s[1]: one tensor twice" % (second, first)


def test_a_16_bit_weight_is_not_its_own_copy():
    at = apart(3)
    at["master"][2] = at["params"][2]
    status, message = call(3, [300] * 3, False, at)
    assert status == N.GDN_ERR_INVALID and message == "master[2] is params[2]: one tensor twice"


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_an_fp32_weight_may_be_its_own_copy(eight):
    """master = [p.float() for p in params] is that, where params are fp32."""
    import torch
    c, d = (adamw.Case(41, [700, 256, 30], ("f32", "bf16", "f32"), eight=eight, master=True) for _ in range(2))
    c.w = [p if p.dtype == torch.float32 else w for p, w in zip(c.p, c.w)]
    c.run(), d.run()
    c.before["w"][0] = c.before["w"][2] = None
    c.w[0] = c.w[2] = None
    c.check()
    for k in ("p", "m", "v"):
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(getattr(c, k), getattr(d, k)))


@pytest.mark.gpu
def test_parts_behind_one_another_are_taken():
    """Flat buffers in any order of their parts, a gradient used twice, and empty tensors anywhere."""
    import torch

    import gated_delta_rule_gate_gb300 as g
    n, size = 80, 100
    order = [(7 * i) % n for i in range(n)]
    flat = [torch.zeros(n * size, device="cuda") for _ in range(3)]
    cut = lambda t: [t[i * size:(i + 1) * size] for i in order]
    grad = torch.ones(size, device="cuda")
    empty = torch.zeros(0, device="cuda")
    p, m, v = (cut(t) + [empty, empty] for t in flat)
    g.gdn_adamw(p, [grad] * n + [empty, empty], m, v, 1, lr=0.5, weight_decay=0.0)
    assert float((flat[0] + 0.5).abs().max()) <= 1e-6
    one = torch.zeros(size, device="cuda")
    for lists, msg in (([p[:2], p[2:4], m[:2], [one, one]], "exp_avg_sq"), ([[one, one], p[:2], m[:2], v[:2]], "params"),
                       ([p[:1], [grad], m[:1], m[:1]], "exp_avg_sq.0. is exp_avg.0.")):
        before = one.clone()
        with pytest.raises(g.GdnError, match=msg):
            g.gdn_adamw(*lists, 1)
        assert torch.equal(one, before)
