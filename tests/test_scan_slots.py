"""Slot ids in calls that hold no states: what the ids may be, and the gradient of a forward
call whose only states were its final ones.  Tolerances as in test_scan.py and
test_scan_backward.py."""
import math

import pytest
import torch

import layer_reference as ref
import test_scan as fwd
import test_scan_backward as bwd
from gated_delta_rule_gate_gb300 import _native as N
from layer_standins import Standin

LENGTHS = [70, 0, 33, 130]


def gradients(p, seed, err, **more):
    import gated_delta_rule_gate_gb300 as g
    c = lambda t: None if t is None else t.cuda()
    kw = dict(beta=c(p["beta"]), gate_bias=c(p["bias"]), gate_scale=c(p["scale"]), beta_sigmoid=True,
              input_scale=p["mode"], cu_seqlens=c(p["cu"]), error_word=err,
              slot_ids=torch.tensor(p["slots"], dtype=torch.int32, device="cuda"))
    x, z = c(p["x"]), c(p["decay"])
    fin = torch.full((p["nrows"], x.shape[1]), math.nan, device="cuda") if p["final"] else None
    out, chunks = g.gdn_scan(x, z, final_state=fin, out=torch.full_like(x, math.nan), want_chunk_states=True, **kw)
    d_out = torch.randn(p["x"].shape, generator=torch.Generator().manual_seed(seed))
    nan = lambda t: torch.full_like(t, math.nan)
    got = g.gdn_scan_backward(c(d_out), x, z, chunks, dx=nan(x), d_decay=nan(z), d_beta=nan(kw["beta"]), **kw, **more)
    return out, fin, d_out, got


@pytest.mark.gpu
@pytest.mark.parametrize("final", [True, False], ids=["final states", "no states"])
def test_gradient_with_slots_beyond_the_batch(final):
    p = fwd.draw(3, 72, lengths=LENGTHS, rows=11, slots=[7, 0, 10, 3], state=False)
    p["final"] = final
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for more in ({}, {"num_state_rows": 11}):
        out, fin, d_out, got = gradients(p, 5, err, **more)
        r_out, r_fin = ref.scan(p)
        assert ref.rel(out, r_out) <= fwd.STATE_TOL
        assert fin is None or ref.rel(fin, r_fin) <= fwd.STATE_TOL
        bwd.check(p, d_out, None, got)
        assert int(err) == 0


@pytest.mark.gpu
def test_slots_that_are_skipped():
    """A negative id without states, and one beyond the rows where their number is known."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = fwd.draw(4, 40, lengths=LENGTHS, rows=100, slots=[70, 1, -1, 3], state=False)
    for final in (False, True):
        p["final"] = final
        out, _, d_out, got = gradients(p, 6, err)
        assert ref.rel(out, ref.scan(p)[0]) <= fwd.STATE_TOL
        assert bool(torch.isnan(out[p["spans"][2][0]:p["spans"][2][1]]).all())
        bwd.check(p, d_out, None, got)
        assert int(err) == N.DEVERR_BAD_SLOT
    p = fwd.draw(4, 40, lengths=LENGTHS, rows=8, slots=[7, 1, 9, 3], state=False)
    p["final"] = True
    _, _, d_out, got = gradients(p, 6, err, num_state_rows=8)
    bwd.check(p, d_out, None, got)


@pytest.mark.gpu
def test_step_with_slots_and_no_states():
    import gated_delta_rule_gate_gb300 as g
    x, z = torch.randn(3, 20, device="cuda"), -torch.rand(3, 20, device="cuda")
    kw = dict(cu_seqlens=torch.arange(4, dtype=torch.int32, device="cuda"))
    slots = torch.tensor([9, 0, 5], dtype=torch.int32, device="cuda")
    assert torch.equal(g.gdn_scan_step(x, z, slot_ids=slots, **kw), g.gdn_scan_step(x, z, **kw))


def test_num_state_rows_is_checked():
    import gated_delta_rule_gate_gb300 as g
    x, ch = Standin((4, 8)), Standin((1, 8))
    for rows in (-1, 0, 2 ** 31, 2 ** 70):
        with pytest.raises(ValueError, match="num_state_rows"):
            g.gdn_scan_backward(x, x, x, ch, num_state_rows=rows)
    with pytest.raises(ValueError, match="num_state_rows"):
        g.gdn_scan_backward(x, x, x, ch, initial_state=Standin((5, 8)), num_state_rows=4)
