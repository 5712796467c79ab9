"""Channel counts that end inside a word, of rows that begin on 16-byte addresses: what lies
behind a row's channels in a wider tensor is neither taken in nor written."""
import math

import pytest
import torch

import layer_reference as ref
import test_scan as fwd
import test_scan_backward as bwd


def widen(t, to, fill):
    wide = torch.full((*t.shape[:-1], to), fill, dtype=t.dtype, device="cuda")
    wide[..., :t.shape[-1]] = t.cuda()
    return wide


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [1, 3, 65, 68, 127, 130])
@pytest.mark.parametrize("layout", [dict(lengths=[300, 1, 199]), dict(S=320, seq_lens=[320, 320])])
def test_rows_with_room_behind_them(act, D, layout):
    import gated_delta_rule_gate_gb300 as g
    p = fwd.draw(D, D, act=act, mode="unit", **layout)
    W = (D + 15) // 8 * 8
    c = lambda t: None if t is None else t.cuda()
    i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")
    x, z, y = (widen(p[k], W, math.nan) for k in ("x", "decay", "beta"))
    kw = dict(gate_bias=c(p["bias"]), gate_scale=c(p["scale"]), beta_sigmoid=True, input_scale="unit",
              cu_seqlens=c(p["cu"]), seq_lens=i32(p["seq_lens"]), initial_state=c(p["h0"]))
    cut = lambda t: t[..., :D]
    out = torch.full_like(x, 7.0)
    _, chunks = g.gdn_scan(cut(x), cut(z), beta=cut(y), out=cut(out), want_chunk_states=True, **kw)
    gen = torch.Generator().manual_seed(1)
    d_out = torch.randn(p["x"].shape, generator=gen).to(p["x"].dtype)
    d = widen(d_out, W, math.nan)
    grads = [torch.full_like(t, 7.0) for t in (x, z, y)]
    got = g.gdn_scan_backward(cut(d), cut(x), cut(z), chunks, beta=cut(y), dx=cut(grads[0]), d_decay=cut(grads[1]),
                              d_beta=cut(grads[2]), **kw)
    for t in [out] + grads:
        assert bool((t[..., D:] == 7.0).all())
    r_out, _ = ref.scan(p)
    assert ref.rel(cut(out), r_out) <= fwd.out_tol(p["x"].dtype)
    bwd.check(p, d_out, None, got)
    step = torch.full_like(x, 7.0)
    g.gdn_scan_step(cut(x), cut(z), beta=cut(y), out=cut(step), **kw)
    assert bool((step[..., D:] == 7.0).all()) and ref.rel(cut(step), r_out) <= fwd.out_tol(p["x"].dtype)
