"""What autograd sees of calls that write into given tensors: their versions move on, so that
a tensor saved for a backward pass and then overwritten is an error."""
import pytest
import torch


def outputs(g):
    """(call, the tensors that it writes)."""
    gen = torch.Generator().manual_seed(2)
    new = lambda *s: torch.randn(*s, generator=gen).cuda()
    x, z, bias, slab, out, fin = new(20, 8), -new(20, 8).abs(), new(8), new(1, 8), new(20, 8), new(1, 8)
    gate = dict(gate_bias=bias, gate_scale=-bias.exp())
    for fn in (g.gdn_scan, g.gdn_scan_step):
        yield lambda fn=fn: fn(x, z, out=out, initial_state=slab, final_state=slab), [out, slab]
        yield lambda fn=fn: fn(x, z, initial_state=slab, final_state=fin), [fin]
    chunks = g.gdn_scan(x, z, beta=x, want_chunk_states=True, **gate)[1]
    d = [new(20, 8), new(20, 8), new(20, 8), new(8), new(8), new(1, 8)]
    yield (lambda: g.gdn_scan_backward(x, x, z, chunks, beta=x, initial_state=slab, dx=d[0], d_decay=d[1], d_beta=d[2],
                                       d_gate_bias=d[3], d_gate_scale=d[4], d_initial_state=d[5], **gate), d)
    res, scales, q = new(20, 8), new(20), torch.empty(20, 8, dtype=torch.float8_e4m3fn, device="cuda")
    yield (lambda: g.gdn_rmsnorm(x, bias, residual=res, residual_out=res, out=q, out_dtype=q.dtype, scales=scales),
           [res, q, scales])
    rstd, dx, dw = g.gdn_rmsnorm(x, bias, want_rstd=True).rstd, new(20, 8), new(8)
    yield lambda: g.gdn_rmsnorm_backward(x, x, bias, rstd, d_residual=dx, dx=dx, d_weight=dw), [dx, dw]
    grads, norm = [new(5), new(7)], new(1)
    yield lambda: g.gdn_grad_clip(grads, 1.0, norm=norm), grads + [norm]
    to = [new(5), new(7)]
    yield lambda: g.gdn_grad_clip(grads, 1.0, out=to), to


@pytest.mark.gpu
def test_given_outputs_get_a_new_version():
    import gated_delta_rule_gate_gb300 as g
    for call, written in outputs(g):
        before = [t._version for t in written]
        call()
        assert [t._version for t in written] == [v + 1 for v in before]
    with torch.inference_mode():  # such tensors have no version
        for call, written in outputs(g):
            call()


@pytest.mark.gpu
def test_a_saved_state_that_is_overwritten_is_noticed():
    import gated_delta_rule_gate_gb300 as g
    x, slab = torch.randn(6, 8, device="cuda"), torch.randn(1, 8, device="cuda")
    w = torch.ones(8, device="cuda", requires_grad=True)
    loss = (slab * w).sum()  # keeps slab
    g.gdn_scan(x, -x.abs(), initial_state=slab, final_state=slab)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
