"""The operators of a block's second half and of its training, run together as they are
used: norm, gated feed-forward, their gradients, the gradients' norm and the AdamW step.

Tolerances.  Between the inputs and a gradient lie at most twelve roundings to the 16-bit
type (the norm's output, the two gates, the output, the products before and behind them, the
same back again), each of them independent from value to value and within one ROUND of it, so
that their squares add up: the norm of all errors is held to twelve ROUNDs of the norm
of the result, which no wrong term would meet.  The AdamW step is held to the formula at the
gradients that came out (its own tests hold each value).
"""
import os
import sys

import pytest
import torch

import layer_reference as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def reference(x, residual, norm, w_gate, w_up, w_down, target):
    """Loss and gradients in 64 bits, by autograd."""
    leaves = [t.detach().double().requires_grad_() for t in (x, residual, norm, w_gate, w_up, w_down)]
    x, residual, norm, w_gate, w_up, w_down = leaves
    r = x + residual
    y = r * (r.square().mean(1, keepdim=True) + 1e-6).rsqrt() * norm
    g = y @ w_gate.T
    out = g * torch.sigmoid(g) * (y @ w_up.T) @ w_down + r
    (out * target.double()).sum().backward()
    return [t.grad for t in leaves]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,D,F", [(300, 256, 512), (77, 72, 131), (9, 128, 200)])
def test_gradients_of_a_block(T, D, F, dt):
    import recurrent_layer as ex
    gen = torch.Generator().manual_seed(T)
    d = ref.DT[dt]
    r = lambda *s: torch.randn(*s, generator=gen)
    x, norm = r(T, D).to(d).cuda(), (1 + 0.1 * r(D)).to(d).cuda()
    residual, target = r(T, D).cuda(), r(T, D).cuda()
    w = [(r(F, D) * k ** -0.5).to(d).cuda() for k in (D, D, F)]
    leaves = [x, residual, norm, *w]
    want = reference(*leaves, target)
    for t in leaves:
        t.requires_grad_()
    y, res = ex.Norm.apply(x, residual, norm)
    out = ex.Glu.apply(y, w[0], w[1]) @ w[2]
    ((res + out.float()) * target).sum().backward()
    for t, g in zip(leaves, want):
        assert float((t.grad.double() - g).norm()) <= 12 * ref.ROUND[d] * float(g.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_training_step_of_a_stack(bits):
    """A step of the example's stack: gradients of every parameter, then the step at them."""
    import recurrent_layer as ex
    stack = ex.Stack(inner=160)
    params = stack.parameters()
    old = [p.clone() for p in params]
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(131, stack.dim, generator=gen, device="cuda").bfloat16()
    for p in params:
        p.requires_grad_()
    stack.train(x, ex.offsets((100, 31))).square().mean().backward()
    grads = [p.grad for p in params]
    assert all(g is not None and bool(g.isfinite().all()) and bool(g.any()) for g in grads)
    kept = [g.clone() for g in grads]
    for p in params:
        p.requires_grad_(False)
    opt = ex.AdamW(params, 1e-2, bits=bits)
    norm = opt.step(grads, 0.5)
    want = sum(float(g.double().square().sum()) for g in kept) ** 0.5
    assert abs(float(norm) - want) <= 1e-5 * want and all(torch.equal(a, b) for a, b in zip(grads, kept))
    k = min(1.0, 0.5 / (float(norm) + 1e-6))
    for p, q, g in zip(params, old, kept):
        g = g.double() * k
        # of the first step m / (1 - beta1) is g and v / (1 - beta2) its square
        step = g / (g.abs() + 1e-8)
        y = q.double() - 1e-2 * (0.01 * q.double() + step)
        r = ref.ROUND[p.dtype]
        assert bool(((p.double() - y).abs() <= r * y.abs() + 2.0 ** -16 * (q.double().abs() + 1e-2)).all())


@pytest.mark.gpu
def test_example_runs():
    """Training by each optimizer, then decode steps that continue the prefill (the bound
    of the plain example, with the two products and norms of the second half besides)."""
    import recurrent_layer as ex
    for optimizer in (ex.AdamW, lambda p, rate: ex.AdamW(p, rate, bits=8)):
        stack = ex.Stack(inner=192)
        losses, norms = ex.train(stack, steps=4, optimizer=optimizer, rate=3e-3)
        assert all(v > 0 and v < float("inf") for v in losses + norms)
        got, want = ex.serve(stack)
        assert float((got - want).abs().max() / want.abs().max()) <= 12 * 2.0 ** -8 + 2.0 ** -4
