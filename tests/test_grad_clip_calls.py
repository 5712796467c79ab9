"""gdn_grad_clip: arguments that are easily left out."""
import pytest
import torch

from layer_standins import Standin


def test_max_norm_is_required():
    import gated_delta_rule_gate_gb300 as g
    for bad in (None, "1"):
        with pytest.raises(TypeError):
            g.gdn_grad_clip([Standin((4,))], bad)
