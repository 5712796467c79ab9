"""gdn_grad_clip: arguments that are easily left out."""
import pytest
import torch

from layer_standins import Standin


def test_max_norm_is_required():
    import gated_delta_rule_gate_gb300 as g
    for bad in (None, "1"):
        with pytest.raises(TypeError):
            g.gdn_grad_clip([Standin((4,))], bad)


@pytest.mark.gpu
def test_a_norm_that_the_call_allocates_belongs_to_its_stream():
    import gated_delta_rule_gate_gb300 as g
    side = torch.cuda.Stream()
    for grads in ([], [torch.ones(5, device="cuda")]):
        torch.cuda.synchronize()
        norm = g.gdn_grad_clip(grads, 1.0, stream=side)
        torch.cuda.synchronize()
        at = norm.data_ptr()
        home = [s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= at < s["address"] + s["total_size"]]
        assert home == [side.cuda_stream]
        assert abs(float(norm) - len(grads) * 5 ** 0.5) < 1e-5
