"""gdn_scan and gdn_scan_step against the token loop in 64 bits, and their refusals.

Tolerances (max |x - ref| / max |ref|).  A token's a = exp(g) carries a relative
error of at most a few 2^-24 (one rounding of g, one of exp, one of the product),
which a state that remembers M tokens sums to M times that; the draws keep
a <= 0.995 (M <= 200), so fp32 states and outputs are held to 200 * 8 * 2^-24 =
1e-4.  An output in 16 bits adds its own rounding.
"""
import ctypes
import math

import pytest
import torch

import layer_reference as ref
from gated_delta_rule_gate_gb300 import _native as N

STATE_TOL = 1e-4
FAKE = 0x100000  # aligned and never read: the call is refused before a launch


def out_tol(dtype):
    return STATE_TOL + ref.ROUND[dtype]


def draw(seed, D, *, lengths=None, S=None, seq_lens=None, cu=None, T=None, act="f32", gate="same", raw=True,
         beta="sigmoid", mode="none", state=True, rows=None, slots=None):
    gen = torch.Generator().manual_seed(seed)
    spans = ref.tokens_of(lengths=lengths, cu=cu, T=T if T is not None else (sum(lengths) if lengths else 0), S=S,
                          seq_lens=seq_lens)
    B = len(spans)
    n = B * S if S is not None else (T if T is not None else sum(lengths))
    lead = (B, S) if S is not None else (n,)
    dt = ref.DT[act]
    gd = dt if gate == "same" else torch.float32
    p = {"mode": mode, "sigmoid": beta == "sigmoid", "spans": spans, "bias": None, "scale": None, "beta": None}
    p["x"] = torch.randn(*lead, D, generator=gen).to(dt)
    if raw:
        p["decay"] = torch.randn(*lead, D, generator=gen).to(gd)
        p["bias"] = torch.rand(D, generator=gen) * 2  # softplus >= 0.05 nearly always
        p["scale"] = -torch.exp(torch.rand(D, generator=gen) * 3 - 2)
    else:
        p["decay"] = (-torch.exp(torch.rand(*lead, D, generator=gen) * 6 - 5.2)).to(gd)  # a <= 0.995
    if beta:
        p["beta"] = torch.randn(*lead, D, generator=gen).to(gd)
    p["nrows"] = rows or B
    p["slots"] = slots
    p["rows"] = [r if 0 <= r < p["nrows"] else None for r in (slots if slots is not None else range(B))]
    p["h0"] = torch.randn(p["nrows"], D, generator=gen) if state else None
    p["S"], p["seq_lens"] = S, seq_lens
    p["cu"] = None
    if S is None:
        off = [0]
        for k in lengths or []:
            off.append(off[-1] + k)
        p["cu"] = torch.tensor(cu if cu is not None else off, dtype=torch.int32)
    return p


def call(p, fn, out=None, fin=None, h0=None, err=None, stream=None, x=None, **kw):
    dev = {k: p[k].cuda() for k in ("x", "decay", "beta", "bias", "scale", "cu") if p[k] is not None}
    i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")
    h0 = h0 if h0 is not None else (p["h0"].cuda() if p["h0"] is not None else None)
    fin = fin if fin is not None else torch.full((p["nrows"], p["x"].shape[-1]), math.nan, device="cuda")
    out = out if out is not None else torch.full(p["x"].shape, math.nan, dtype=p["x"].dtype, device="cuda")
    fn(dev["x"] if x is None else x, dev["decay"], beta=dev.get("beta"), gate_bias=dev.get("bias"),
       gate_scale=dev.get("scale"), beta_sigmoid=p["sigmoid"] and p["beta"] is not None, input_scale=p["mode"],
       cu_seqlens=dev.get("cu"), seq_lens=i32(p["seq_lens"]), slot_ids=i32(p["slots"]), initial_state=h0,
       final_state=fin, out=out, error_word=err, stream=stream, **kw)
    return out, fin


def check(p, out, fin):
    r_out, r_fin = ref.scan(p)
    assert ref.rel(out, r_out) <= out_tol(p["x"].dtype)
    assert ref.rel(fin, r_fin) <= STATE_TOL
    D = p["x"].shape[-1]
    # tokens of no request and rows of none keep what was there
    assert bool(torch.isnan(out.float().cpu().reshape(-1, D)[torch.isnan(r_out)]).all())
    assert bool(torch.isnan(fin.cpu()[torch.isnan(r_fin)]).all())


def both():
    import gated_delta_rule_gate_gb300 as g
    return [g.gdn_scan, g.gdn_scan_step]


CASES = [
    dict(D=1, lengths=[1]),
    dict(D=2, lengths=[3, 0, 1], mode="unit"),
    dict(D=63, lengths=[0, 0, 130, 1, 0, 17, 0], mode="lerp"),
    dict(D=64, lengths=[128, 128], raw=False, beta=None),
    dict(D=65, lengths=[16, 15, 17, 1, 1, 1, 300], act="f16", mode="unit"),
    dict(D=130, lengths=[700], act="bf16", raw=False, mode="lerp"),
    dict(D=130, lengths=[64] * 9, act="f16", gate="f32", beta="plain"),
    dict(D=200, lengths=[1] * 40, act="bf16", gate="f32", raw=False, beta=None),
    dict(D=34, lengths=[2500, 1, 2600], act="f16", mode="unit"),
    dict(D=8, lengths=[4100, 33], beta=None, state=False),
    dict(D=96, S=70, seq_lens=[70, 0, 1, 69, 33], act="f16", mode="unit"),
    dict(D=10, S=5, seq_lens=[5, -3, 2, 9, 0, 1]),  # clamped to [0, S]
    dict(D=40, cu=[-5, 20, 20, 61, 900], T=77, act="bf16"),  # offsets clamped to [0, T], a gap before none
    dict(D=40, cu=[7, 20, 20, 50], T=77),  # tokens of no request at both ends
    dict(D=72, lengths=[5, 40, 0, 9], rows=11, slots=[7, 0, 10, 3], mode="lerp"),
    dict(D=72, lengths=[5, 40, 0, 9], rows=4, slots=[3, -1, 4, 0], act="f16"),  # two bad slots
    # equal rows, which a cluster shares out in groups of requests
    dict(D=70, S=600, seq_lens=[600, 599, 0, 300], act="f16", mode="unit"),
    dict(D=130, S=321, seq_lens=[321] * 8, mode="lerp"),
    dict(D=34, S=1100, seq_lens=[1100, 1], act="bf16", rows=3, slots=[2, 0]),
    dict(D=66, S=2048, seq_lens=[2048, 2047, 2048], act="f16", gate="f32", beta="plain"),
]


def lens_clamped(c):
    if c.get("seq_lens"):
        c = dict(c, seq_lens=[min(max(n, 0), c["S"]) for n in c["seq_lens"]])
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_the_token_loop(i):
    c = CASES[i]
    p = draw(100 + i, **lens_clamped(c))
    if c.get("seq_lens"):
        p["seq_lens"] = c["seq_lens"]
    for fn in both():
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, fin = call(p, fn, err=err)
        check(p, out, fin)
        assert int(err) == (N.DEVERR_BAD_SLOT if None in p["rows"] else 0)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("layout", [dict(lengths=[300, 0, 1, 399]), dict(S=350, seq_lens=[350, 349])])
def test_wide_rows_in_several_windows(act, layout):
    """So many channels that few blocks walk each: several windows, with the blocks of a
    pass that keeps states and of one that does not."""
    import gated_delta_rule_gate_gb300 as g
    p = draw(250, 8192, act=act, mode="unit", **layout)
    for keep in (False, True):
        out, fin = call(p, g.gdn_scan, want_chunk_states=keep)
        check(p, out, fin)
        again = call(p, g.gdn_scan, want_chunk_states=keep)
        assert torch.equal(out.nan_to_num(9.0), again[0].nan_to_num(9.0)) and torch.equal(fin, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("mode", ["none", "lerp", "unit"])
@pytest.mark.parametrize("raw", [True, False])
def test_types_and_gates(act, mode, raw):
    for k, beta in enumerate([None, "plain", "sigmoid"]):
        p = draw(300 + k, 150, lengths=[200, 1, 0, 333], act=act, mode=mode, raw=raw, beta=beta,
                 gate="f32" if k == 1 else "same")
        for fn in both():
            check(p, *call(p, fn))


@pytest.mark.gpu
def test_slab_in_place_and_resume():
    """One request run in three pieces through a slab updated in place equals one run."""
    import gated_delta_rule_gate_gb300 as g
    p = draw(7, 192, lengths=[1000], act="f16", mode="unit", rows=5, slots=[3])
    whole_out, whole_fin = call(p, g.gdn_scan)
    slab = p["h0"].cuda()
    before = slab.clone()
    outs = []
    for a, b, fn in ((0, 511, g.gdn_scan), (511, 998, g.gdn_scan), (998, 1000, g.gdn_scan_step)):
        q = dict(p, x=p["x"][a:b], decay=p["decay"][a:b], beta=p["beta"][a:b],
                 cu=torch.tensor([0, b - a], dtype=torch.int32))
        outs.append(call(q, fn, fin=slab, h0=slab)[0])
    assert ref.rel(torch.cat(outs), whole_out.double().cpu()) <= 2 * out_tol(torch.float16)
    assert ref.rel(slab[3], whole_fin[3].double().cpu()) <= 2 * STATE_TOL
    keep = [0, 1, 2, 4]
    assert torch.equal(slab[keep], before[keep])


@pytest.mark.gpu
def test_a_request_does_not_see_its_neighbours():
    """NaN and infinities inside one request, in its state and in the tokens of no
    request reach no other request."""
    for S in (None, 90):
        kw = dict(lengths=[40, 90, 61, 300]) if S is None else dict(S=90, seq_lens=[40, 90, 61, 5])
        p = draw(11, 70, act="f32", mode="lerp", **kw)
        r_out, r_fin = ref.scan(p)
        q = dict(p, x=p["x"].clone(), decay=p["decay"].clone(), h0=p["h0"].clone())
        t0, t1 = p["spans"][1]
        X, Z = q["x"].reshape(-1, 70), q["decay"].reshape(-1, 70)
        X[t0 + 3] = math.nan
        X[t1 - 1] = math.inf
        Z[t0 + 50] = math.inf
        q["h0"][1] = math.nan
        if S is not None:
            used = torch.zeros(X.shape[0], dtype=torch.bool)
            for a, b in p["spans"]:
                used[a:b] = True
            X[~used] = math.nan
            Z[~used] = math.nan
        for fn in both():
            out, fin = call(q, fn)
            out = out.reshape(-1, 70)
            for b in (0, 2, 3):
                a, e = p["spans"][b]
                assert ref.rel(out[a:e], r_out[a:e]) <= STATE_TOL
                assert ref.rel(fin[b], r_fin[b]) <= STATE_TOL


@pytest.mark.gpu
def test_extreme_gates():
    """g = 0 keeps everything (a running sum), g = -inf forgets the past, LERP and
    UNIT then pass the input on or drop it."""
    T, D = 600, 66
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(5))
    for mode in ("none", "lerp", "unit"):
        z = torch.zeros(T, D)
        z[:, 1::3] = -math.inf
        p = {"x": x, "decay": z, "beta": None, "bias": None, "scale": None, "mode": mode, "sigmoid": False,
             "spans": [(0, T)], "rows": [0], "nrows": 1, "h0": torch.randn(1, D), "slots": None, "seq_lens": None,
             "S": None, "cu": None}
        r_out, _ = ref.scan(p)
        for fn in both():
            out, _ = call(p, fn)
            # 600 additions in fp32: 600 * 2^-24 relative to the largest partial sum
            assert ref.rel(out, r_out) <= 600 * 2.0 ** -24


@pytest.mark.gpu
def test_columns_of_a_wider_matrix():
    """x, decay, beta and out as column slices, at even and odd offsets, of one
    matrix with a token stride of its own."""
    import gated_delta_rule_gate_gb300 as g
    for off in (0, 1, 2, 4):
        for lead in ((150,), (3, 50)):
            D = 68
            wide = torch.randn(*lead, 4 * D + 8, generator=torch.Generator().manual_seed(off)).half().cuda()
            x, z, y = (wide[..., off + k * D:off + (k + 1) * D] for k in range(3))
            o = torch.zeros(*lead, 2 * D + off + 4, dtype=torch.half, device="cuda")
            scale = -torch.rand(D, device="cuda")
            bias = torch.rand(D, device="cuda")
            for fn in both():
                got = fn(x, z, beta=y, gate_bias=bias, gate_scale=scale, beta_sigmoid=True, input_scale="unit",
                         out=o[..., off:off + D])
                want = fn(x.contiguous(), z.contiguous(), beta=y.contiguous(), gate_bias=bias, gate_scale=scale,
                          beta_sigmoid=True, input_scale="unit")
                assert torch.equal(got, want)
                assert not bool(o[..., off + D:].any()) and not bool(o[..., :off].any())
                o.zero_()
    assert g.gdn_scan(torch.empty(0, 8, device="cuda"), torch.empty(0, 8, device="cuda")).shape == (0, 8)


@pytest.mark.gpu
def test_same_bits_on_every_run_and_any_stream():
    p = draw(21, 2048, lengths=[3000, 77, 1500], act="bf16", mode="unit")
    import gated_delta_rule_gate_gb300 as g
    first = call(p, g.gdn_scan)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream):
        out, fin = call(p, g.gdn_scan, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(fin, first[1])
    # outputs allocated by the call belong to the stream of the call
    got = g.gdn_scan(p["x"].cuda(), p["decay"].cuda(), stream=side)
    side.synchronize()
    assert torch.equal(got, g.gdn_scan(p["x"].cuda(), p["decay"].cuda()))


@pytest.mark.gpu
def test_decreasing_offsets_are_reported():
    p = draw(31, 32, cu=[0, 30, 20, 40], T=40)
    for fn in both():
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(p, fn, err=err)
        torch.cuda.synchronize()
        assert int(err) == N.DEVERR_OVERLAP


def _args(**over):
    a = N.GdnScanArgs(2, 8, 0, 16, 0, N.DTYPE_F16, N.DTYPE_F16, 0, 0, 0, 0, 0, 0, FAKE, FAKE, None, FAKE)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status,msg", [
    (dict(batch=-1), N.GDN_ERR_INVALID, "batch"),
    (dict(total_tokens=-1), N.GDN_ERR_INVALID, "total_tokens"),
    (dict(channels=0), N.GDN_ERR_INVALID, "channels"),
    (dict(channels=(1 << 24) + 1), N.GDN_ERR_UNSUPPORTED, "2^24"),
    (dict(act_dtype=3), N.GDN_ERR_INVALID, "dtype"),
    (dict(gate_dtype=N.DTYPE_BF16), N.GDN_ERR_INVALID, "gate_dtype"),
    (dict(input_scale=3), N.GDN_ERR_INVALID, "input_scale"),
    (dict(flags=N.FLAG_L2NORM_Q), N.GDN_ERR_INVALID, "flag"),
    (dict(flags=N.FLAG_BETA_SIGMOID), N.GDN_ERR_INVALID, "without beta"),
    (dict(seq_len=4, cu_seqlens=FAKE), N.GDN_ERR_INVALID, "packed"),
    (dict(seq_len=3), N.GDN_ERR_INVALID, "batch * seq_len"),
    (dict(seq_lens=FAKE), N.GDN_ERR_INVALID, "uniform form"),
    (dict(total_tokens=7), N.GDN_ERR_INVALID, "multiple of batch"),
    (dict(gate_bias=FAKE), N.GDN_ERR_INVALID, "together"),
    (dict(gate_scale=FAKE), N.GDN_ERR_INVALID, "together"),
    (dict(num_state_rows=1), N.GDN_ERR_INVALID, "num_state_rows"),
    (dict(num_state_rows=-1), N.GDN_ERR_INVALID, "num_state_rows"),
    (dict(x=None), N.GDN_ERR_INVALID, "required"),
    (dict(o=None), N.GDN_ERR_INVALID, "required"),
    (dict(x=FAKE + 1), N.GDN_ERR_INVALID, "aligned"),
    (dict(initial_state=FAKE + 2), N.GDN_ERR_INVALID, "aligned"),
    (dict(x_stride=15), N.GDN_ERR_INVALID, "x_stride"),
    (dict(o_stride=-16), N.GDN_ERR_INVALID, "o_stride"),
])
def test_refuses(over, status, msg):
    for fn in (N.load().gdn_scan, N.load().gdn_scan_step):
        assert fn(ctypes.byref(_args(**over)), None) == status
        assert msg.lower() in N.last_error_message().lower()


def test_refuses_chunk_states_in_the_step_and_takes_no_requests():
    lib = N.load()
    assert lib.gdn_scan_step(ctypes.byref(_args(chunk_states=FAKE)), None) == N.GDN_ERR_INVALID
    assert lib.gdn_scan(None, None) == N.GDN_ERR_INVALID
    assert lib.gdn_scan(ctypes.byref(_args(batch=0, total_tokens=0)), None) == N.GDN_OK  # nothing to launch


def test_binding_refuses():
    import gated_delta_rule_gate_gb300 as g
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device"):
        g.gdn_scan(x, x)
    with pytest.raises(TypeError, match="dtype"):
        g.gdn_scan(x.double(), x)
    with pytest.raises(ValueError, match="tokens, channels"):
        g.gdn_scan(x[0], x[0])
    with pytest.raises(ValueError, match="input_scale"):
        g.gdn_scan(x, x, input_scale="sqrt")
    with pytest.raises(ValueError, match="packed"):
        g.gdn_scan(x[None], x[None], cu_seqlens=torch.zeros(2, dtype=torch.int32))
