"""gdn_glu where the activation is far in its tail.

With weights [inner, 1] and tokens of 1 the gates are the weights themselves, without an error, so that
out = act(g) u has that of the activation alone: within (8 + |z| + g^2) 2^-22 of its value, z the
argument of the exponential, and the rounding of the type.  Beyond |z| = 87 the exponential and what
multiplies g are no normal fp32 numbers, but come in steps of 2^-149: a step for the exponential, and half
a step for each of the two products behind it."""
import pytest
import torch

import layer_reference as ref
import test_glu as glu


def act(g, kind):
    """As in test_glu; of "gelu" by erfc, which keeps its digits in the tail."""
    a, slope, z = glu.act(g, kind)
    return (g * 0.5 * torch.special.erfc(-g * 0.5 ** 0.5) if kind == "gelu" else a), slope, z


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("kind", ["silu", "sigmoid", "gelu_tanh", "gelu"])
def test_where_the_exponential_is_near_its_smallest(kind, T):
    import gated_delta_rule_gate_gb300 as gdn
    # of the exponential's argument: silu and sigmoid take g itself; the others reach 89 at smaller g
    least = {"silu": 89.0, "sigmoid": 89.0, "gelu_tanh": 10.0625, "gelu": 13.3125}[kind]
    g = torch.linspace(-least, -least / 2, 600).bfloat16()
    _, _, z = act(g.double(), kind)
    assert 88 <= float((g.double() ** 2 / 2 if kind == "gelu" else z.abs()).max()) <= 89.2
    u = torch.full_like(g, 2.0 ** 120)
    x = torch.ones(T, 1, dtype=torch.bfloat16, device="cuda")
    wg, wu = g[:, None].cuda(), u[:, None].cuda()
    out, gates = gdn.gdn_glu(x, wg, wu, activation=kind, want_gates=True)
    kept = glu.unpack(gates, 600)
    assert bool((kept[:, 0] == g.cuda().float()).all()) and bool((kept[:, 1] == 2.0 ** 120).all())
    a, _, z = act(g.double().cuda(), kind)
    want = a * 2.0 ** 120
    tol = glu.fuzz(g.double().cuda(), z) * want.abs() + 2 * 2.0 ** -149 * g.double().cuda().abs() * 2.0 ** 120
    tol = tol + ref.ROUND[torch.bfloat16] * (want.abs() + tol)
    assert bool(((out.double() - want).abs() <= tol).all())
    assert bool((out == gdn.gdn_glu(x, wg, wu, activation=kind)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("kind", ["silu", "sigmoid", "gelu_tanh", "gelu", "relu"])
def test_nan_and_the_largest_gates(kind, T):
    """A NaN stays one, a large gate is itself or 0 behind the activation."""
    import gated_delta_rule_gate_gb300 as gdn
    g = torch.tensor([float("nan"), 1e30, -1e30, 200.0, -200.0, 30.0, 31.0]).bfloat16()
    x = torch.ones(T, 1, dtype=torch.bfloat16, device="cuda")
    out = gdn.gdn_glu(x, g[:, None].cuda(), torch.ones(7, 1, dtype=torch.bfloat16, device="cuda"), activation=kind)
    big = (lambda v: 1.0) if kind == "sigmoid" else (lambda v: v)
    assert bool(out[:, 0].isnan().all())
    for i in (1, 3, 5, 6):
        assert bool((out[:, i] == big(float(g[i]))).all())
    for i in (2, 4):
        assert bool((out[:, i] == 0).all())
