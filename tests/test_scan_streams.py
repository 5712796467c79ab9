"""gdn_scan and gdn_scan_backward on a stream of their own, which waits for what fills their
tensors: the same bits as on the current one."""
import math

import pytest
import torch

import test_scan as fwd


@pytest.mark.gpu
@pytest.mark.parametrize("D", [1100, 1024])
def test_same_bits_on_a_stream_that_waits(D):
    import gated_delta_rule_gate_gb300 as g
    p = fwd.draw(61, D, lengths=[3000, 77, 1500], act="bf16", mode="unit")
    c = lambda t: t.cuda()
    x, z = c(p["x"]), c(p["decay"])
    d_out = torch.randn(p["x"].shape, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    kw = dict(beta=c(p["beta"]), gate_bias=c(p["bias"]), gate_scale=c(p["scale"]), beta_sigmoid=True,
              input_scale="unit", cu_seqlens=c(p["cu"]), initial_state=c(p["h0"]))
    side, first = torch.cuda.Stream(), None
    for turn in range(12):
        stream = side if turn % 2 else torch.cuda.current_stream()
        nan = lambda t: torch.full_like(t, math.nan)
        given = dict(dx=nan(x), d_decay=nan(z), d_beta=nan(x), d_initial_state=nan(kw["initial_state"]))
        out = nan(x)
        side.wait_stream(torch.cuda.current_stream())
        _, chunks = g.gdn_scan(x, z, out=out, want_chunk_states=True, stream=stream, **kw)
        got = g.gdn_scan_backward(d_out, x, z, chunks, stream=stream, **given, **kw)
        torch.cuda.current_stream().wait_stream(side)
        res = [t.clone() for t in (out, *got)]
        torch.cuda.synchronize()
        first = first or res
        assert all(torch.equal(a, b) for a, b in zip(first, res))
