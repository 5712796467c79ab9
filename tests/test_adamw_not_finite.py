"""gdn_adamw where gradients are not finite or their squares beyond fp32, and the codes of 8-bit
states, in whole rows of 256 elements and in rows at odd addresses."""
import math

import pytest
import torch

from test_adamw import BLOCK, HYPER, U, Case


def states(c, i=0):
    """m and what exp_avg_sq holds (v, or its root in 8 bits) of tensor i."""
    m, v = c.m[i].float(), c.v[i].float()
    if c.eight:
        n = m.numel()
        m = m * c.ms[i].repeat_interleave(BLOCK)[:n]
        v = v * c.vs[i].repeat_interleave(BLOCK)[:n]
    return m, v


@pytest.mark.gpu
@pytest.mark.parametrize("at", [0, 3])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_gradient_that_is_not_finite_marks_its_block(bad, at):
    """With 8-bit states both states of its block of 256 are NaN, whose scales say so; every
    other block is what it is without that gradient."""
    n, hit = 5 * BLOCK + 77, (BLOCK + 9, 5 * BLOCK + 70)
    for where in hit:
        c, d = (Case(31, [n], eight=True, at=at) for _ in range(2))
        c.g[0][where] = bad
        c.run(), d.run()
        block = torch.zeros(n, dtype=torch.bool, device="cuda")
        b = where // BLOCK
        block[b * BLOCK:(b + 1) * BLOCK] = True
        for (y, z), scales in zip(zip(states(c), states(d)), (c.ms[0], c.vs[0])):
            assert bool(y[block].isnan().all()) and torch.equal(y[~block], z[~block])
            assert not bool(scales[b].isfinite())
        assert torch.equal(c.p[0][~block], d.p[0][~block])
        # the step itself is taken before the states are codes: its neighbours move as they would
        rest = torch.arange(n, device="cuda") != where
        assert torch.equal(c.p[0][rest], d.p[0][rest])


@pytest.mark.gpu
@pytest.mark.parametrize("at", [0, 3])
def test_a_gradient_that_is_not_finite_stays_by_itself_in_32_bits(at):
    for bad in (math.inf, math.nan):
        c, d = (Case(32, [700], at=at) for _ in range(2))
        c.g[0][300] = bad
        c.run(), d.run()
        rest = torch.arange(700, device="cuda") != 300
        for k in ("p", "m", "v"):
            assert torch.equal(getattr(c, k)[0][rest], getattr(d, k)[0][rest])
        assert not bool(c.m[0][300].isfinite()) and not bool(c.v[0][300].isfinite())


@pytest.mark.gpu
@pytest.mark.parametrize("at", [0, 3])
def test_a_square_beyond_fp32(at):
    """g = 2^70 squares to an infinite v: exp_avg_sq's block is NaN, exp_avg's is as ever, and the
    parameter takes m / inf = 0 beside its decay."""
    n, where = 600, 300
    c = Case(33, [n], eight=True, at=at)
    c.g[0][where] = 2.0 ** 70
    before = c.p[0].clone()
    c.run()
    m, r = states(c)
    inside = slice(BLOCK, 2 * BLOCK)
    assert bool(m.isfinite().all()) and bool(r[inside].isnan().all())
    assert bool(r[:BLOCK].isfinite().all()) and bool(r[2 * BLOCK:].isfinite().all())
    # m of 0.1 2^70 is the block's largest: the code 448 of a scale that is it / 448
    assert abs(float(m[where]) / (0.1 * 2.0 ** 70) - 1) <= 2.0 ** -20
    want = float(before[where]) * (1 - HYPER["lr"] * HYPER["weight_decay"])
    assert abs(float(c.p[0][where]) - want) <= 4 * U * abs(want)


@pytest.mark.gpu
@pytest.mark.parametrize("at", [0, 3])
def test_codes_are_those_of_the_formula_at_any_address(at):
    """To the bit, as for whole rows, with a short last block."""
    n = 40 * BLOCK + 100
    c = Case(34, [n], eight=True, at=at)
    m, v, ms, vs = (t[0].clone() for t in (c.m, c.v, c.ms, c.vs))
    c.run()
    g, blocks = c.g[0], -(-n // BLOCK)
    spread = lambda s: s.repeat_interleave(BLOCK)[:n]
    m32 = HYPER["beta1"] * (m.float() * spread(ms)) + (1 - HYPER["beta1"]) * g
    v32 = HYPER["beta2"] * (v.float() * spread(vs)).square() + (1 - HYPER["beta2"]) * g.square()
    for y, codes, scales, root in ((m32, c.m[0], c.ms[0], False), (torch.sqrt(v32), c.v[0], c.vs[0], True)):
        pad = torch.zeros(blocks * BLOCK, device="cuda")
        pad[:n] = y
        s = torch.clamp(pad.view(blocks, BLOCK).abs().amax(1), min=2.0 ** -100) * (1 / 448)
        q = y / spread(s)
        if root:
            q = torch.where(q > 0, torch.clamp(q, min=2.0 ** -9), q)
        assert torch.equal(q.to(torch.float8_e4m3fn).view(torch.uint8), codes.view(torch.uint8))
        assert torch.equal(s, scales)
