"""gdn_glu_backward sums each gradient in the order that the sizes decide: which of the
gradients are wanted has no say in their bits.  Sizes at which one gradient, the other or
both are summed over stretches of K."""
import pytest
import torch

import layer_reference as ref


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,D,F", [(1280, 64, 1280), (1001, 517, 1531), (4096, 512, 1536), (1536, 96, 768), (768, 64, 768),
                                   (1000, 64, 768)])
def test_bits_of_a_gradient_do_not_depend_on_the_others(T, D, F, dt):
    import gated_delta_rule_gate_gb300 as gdn
    gen = torch.Generator().manual_seed(T)
    draw = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(ref.DT[dt]).cuda()
    x, wg, wu, d = draw(T, D), draw(F, D, std=D ** -0.5), draw(F, D, std=D ** -0.5), draw(T, F)
    _, gates = gdn.gdn_glu(x, wg, wu, want_gates=True)
    all_of = gdn.gdn_glu_backward(d, x, wg, wu, gates)
    only_x = gdn.gdn_glu_backward(d, x, wg, wu, gates, want_d_weights=False)
    only_w = gdn.gdn_glu_backward(d, x, wg, wu, gates, want_dx=False)
    assert torch.equal(only_x.dx, all_of.dx)
    assert torch.equal(only_w.d_w_gate, all_of.d_w_gate) and torch.equal(only_w.d_w_up, all_of.d_w_up)
