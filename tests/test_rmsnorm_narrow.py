"""The gradient of the norm on rows of a few values against differences of the 64-bit forward
pass, value for value.

Tolerance.  dx is the gradient for the rstd that it is given, which is fp32: off by at most
d = 2^-22 (two last places of rsqrtf) and (dim + 3) 2^-25 (the sum, its mean) of itself.
d dx / d rstd = weight d_out - 3 xhat mean(weight d_out xhat), at most (1 + 3 sqrt(dim)) of the
largest |weight d_out|, so dx is off by rstd d times that, and by 2^-23 of rstd |weight d_out|
for its own rounding.  On rows of one value all but eps / (r^2 + eps) of dx cancels, and what is
left may be smaller than this: it is no more than rstd's digits give."""
import pytest
import torch


@pytest.mark.gpu
@pytest.mark.parametrize("eps", [1e-6, 1e-2])
@pytest.mark.parametrize("D", [1, 2, 7, 31])
def test_differences_value_for_value(D, eps):
    import gated_delta_rule_gate_gb300 as g
    gen = torch.Generator().manual_seed(D)
    n = 60
    x, d_out = torch.randn(n, D, generator=gen), torch.randn(n, D, generator=gen)
    w = 1 + 0.3 * torch.randn(D, generator=gen)
    f = g.gdn_rmsnorm(x.cuda(), w.cuda(), eps=eps, want_rstd=True)
    dx = g.gdn_rmsnorm_backward(d_out.cuda(), x.cuda(), w.cuda(), f.rstd).dx.double().cpu()

    def loss(r):  # of each row
        rstd = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + eps)
        return (r * rstd * w.double() * d_out.double()).sum(1)

    step = 1e-6
    wd = (w.double() * d_out.double()).abs()
    rstd = f.rstd.double().cpu()
    d = 2.0 ** -22 + (D + 3) * 2.0 ** -25
    for j in range(D):
        way = torch.zeros(n, D, dtype=torch.double)
        way[:, j] = step
        diff = (loss(x.double() + way) - loss(x.double() - way)) / (2 * step)
        # the differences: 1e-16 / step of the row's loss, step^2 of the third derivative (at most 15 rstd^3 of it)
        own = 1e-9 * rstd * wd.sum(1) + 15 * step ** 2 * rstd ** 3 * wd.sum(1)
        tol = rstd * (d * (1 + 3 * D ** 0.5) * wd.amax(1) + 2.0 ** -23 * wd[:, j]) + own
        assert bool(((dx[:, j] - diff).abs() <= tol).all())
