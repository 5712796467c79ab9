"""The recurrent-layer operators captured in a CUDA graph: the replay computes what the calls do.

Every kernel sums in a fixed order, so the two results are the same bits.
"""
import pytest
import torch


def layer(g, t, slab):
    """One pass of all operators; `slab` is stepped in place."""
    n = g.gdn_rmsnorm(t["x"], t["w"], residual=t["res"], want_rstd=True)
    kw = dict(beta=t["y"], beta_sigmoid=True, gate_bias=t["bias"], gate_scale=t["scale"], input_scale="unit",
              cu_seqlens=t["cu"])
    out, chunks = g.gdn_scan(n.out, t["z"], want_chunk_states=True, **kw)
    s = g.gdn_scan_backward(t["d"], n.out, t["z"], chunks, **kw)
    b = g.gdn_rmsnorm_backward(s.dx, n.residual, t["w"], n.rstd, d_residual=t["res"])
    clipped = [torch.empty_like(v) for v in (b.dx, s.d_decay, b.dweight)]
    norm = g.gdn_grad_clip([b.dx, s.d_decay, b.dweight], 0.1, out=clipped)
    step = g.gdn_scan_step(t["x"][:3], t["z"][:3], gate_bias=t["bias"], gate_scale=t["scale"], cu_seqlens=t["ones"],
                           initial_state=slab, final_state=slab)
    return [n.out, out, s.d_beta, s.d_gate_bias, s.d_gate_scale, norm, step, *clipped]


@pytest.mark.gpu
@pytest.mark.parametrize("T, D", [(50, 40), (700, 264), (3000, 130)])
def test_replay_computes_what_the_calls_do(T, D):
    import gated_delta_rule_gate_gb300 as g
    gen = torch.Generator().manual_seed(T)
    draw = lambda *s: torch.randn(*s, generator=gen)
    bf = lambda *s: draw(*s).bfloat16().cuda()
    t = {"x": bf(T, D), "z": bf(T, D), "y": bf(T, D), "d": bf(T, D), "w": bf(D), "res": draw(T, D).cuda(),
         "bias": draw(D).cuda(), "scale": -draw(D).exp().cuda(),
         "cu": torch.tensor([0, T // 3, T], dtype=torch.int32).cuda(),
         "ones": torch.arange(4, dtype=torch.int32).cuda()}
    slab = torch.zeros(3, D, device="cuda")
    for _ in range(2):
        want = layer(g, t, slab)
    after = slab.clone()
    slab.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(g, t, slab)
    for v in got:
        v.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(slab, after)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
