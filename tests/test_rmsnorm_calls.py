"""gdn_rmsnorm: arguments that go together."""
import pytest

from layer_standins import Standin


def test_residual_out_without_a_residual_is_refused():
    import gated_delta_rule_gate_gb300 as g
    x, w = Standin((6, 8)), Standin((8,))
    with pytest.raises(ValueError, match="residual_out"):
        g.gdn_rmsnorm(x, w, residual_out=x)
