"""gdn_adamw with an eps that is no normal fp32 number."""
import pytest
import torch

from test_adamw import HYPER, U, Case


@pytest.mark.gpu
@pytest.mark.parametrize("eps", [1e-38, 1e-40, 2.0 ** -149, 1e-60])
@pytest.mark.parametrize("eight", [False, True])
def test_an_eps_below_the_normal_numbers(eight, eps):
    """Where nothing was ever learnt (zero gradients and states) nothing moves but by the decay;
    elsewhere the step is that of the formula."""
    for at in (0, 3):
        c = Case(35, [1000], eight=eight, fresh=True, at=at)
        c.g[0][:600] = 0
        c.before["g"] = [c.g[0].clone()]
        old = c.p[0].clone()
        c.run(1, eps=eps)
        want = old[:600].double() * (1 - HYPER["lr"] * HYPER["weight_decay"])
        assert bool(((c.p[0][:600].double() - want).abs() <= 4 * U * want.abs()).all())
        if eps >= 2.0 ** -149:
            c.check(1, eps=eps)


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_a_small_eps_divides(eight):
    """m that is left where v has come to nothing: m / eps, eps no normal number."""
    c = Case(36, [300], eight=eight, fresh=True)
    c.g[0].zero_()
    if eight:
        c.ms[0].fill_(2.0 ** -120)
        c.m[0].copy_(torch.full((300,), 16.0, device="cuda").to(torch.float8_e4m3fn))
    else:
        c.m[0].fill_(2.0 ** -116)
    old = c.p[0].clone()
    eps, t = 2.0 ** -130, 3
    c.run(t, eps=eps, weight_decay=0.0, lr=1e-6)
    step = 1e-6 / (1 - HYPER["beta1"] ** t) * (HYPER["beta1"] * 2.0 ** -116 / eps)
    want = old.double() - step
    assert bool(((c.p[0].double() - want).abs() <= 16 * U * (abs(step) + want.abs() + old.double().abs())).all())
