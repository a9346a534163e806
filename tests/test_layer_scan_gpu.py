"""GPU parity of the element-wise gated recurrence (lattice_osr_scan_*) against
the fp64 oracle (oracle/layer.py), element by element.

Bars: the oracle's own bounds (every fp32 rounding counted at the magnitude of
its operands, hardware 2^x, 1/x and roots at two units), plus half a step of a
bf16 output (2^-8 of the value).
"""
import math

import pytest
import torch

from compressed_memory_linear_amd import osr
from oracle import layer

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
WEIGHTS = [osr.SCAN_ONE, osr.SCAN_COMPLEMENT, osr.SCAN_NORM]


def make(B, T, D, dtype=BF, gamma=True, seed=0, mean=2.0, state=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, m=0.0: torch.randn(s, generator=g, device="cuda") + m
    return dict(v=r(B, T, D).to(dtype), mu_logit=r(B, T, D, m=mean).to(dtype),
                gamma_logit=r(B, T, D).to(dtype) if gamma else None, state_in=r(B, D) if state else None)


def grads_of(B, T, D, y_dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    return (torch.randn((B, T, D), generator=g, device="cuda").to(y_dtype),
            torch.randn((B, D), generator=g, device="cuda"))


def check(name, got, ref, bound):
    err = (got.double() - ref).abs()
    lim = layer.rounded(bound, ref, got.dtype)
    assert torch.isfinite(got).all(), name
    worst = float((err / lim).max()) if err.numel() else 0.0
    print(f"  {name}: worst error / bar {worst:.3f}", flush=True)
    assert worst <= 1.0, (name, worst)


def oracle(x, weight, lengths=None, dy=None, dso=None):
    return layer.scan(x["v"], x["mu_logit"], x["gamma_logit"], x["state_in"], lengths, weight, dy, dso)


def run_all(x, weight, lengths=None, y_dtype=F, grad_dtype=F, seed=0):
    B, T, D = x["v"].shape
    print(f"scan B{B} T{T} D{D} {x['v'].dtype} y {y_dtype} grad {grad_dtype} weight {weight} "
          f"gamma {x['gamma_logit'] is not None} lengths {lengths is not None}", flush=True)
    dy, dso = grads_of(B, T, D, y_dtype, seed)
    kw = dict(gamma_logit=x["gamma_logit"], lengths=lengths, input_weight=weight)
    y, st, saved = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], y_dtype=y_dtype, save=True, **kw)
    y2, st2 = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], y_dtype=y_dtype, **kw)
    g = osr.lattice_osr_scan_bwd(x["v"], x["mu_logit"], dy, dso, saved=saved, grad_dtype=grad_dtype, **kw)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(st, st2)
    out, bound = oracle(x, weight, lengths, dy, dso)
    got = dict(g, y=y, state_out=st)
    for n in got:
        check(n, got[n], out[n], bound[n])
    return got


SHAPES = [(1, 1, 1), (2, 3, 5), (1, 1, 64), (3, 127, 64), (2, 128, 66), (2, 129, 130), (1, 1000, 257), (5, 260, 128),
          (1, 3001, 192), (40, 17, 24), (2, 511, 1000)]


@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F])
def test_shapes(B, T, D, dtype):
    run_all(make(B, T, D, dtype, seed=T), osr.SCAN_COMPLEMENT, y_dtype=dtype, grad_dtype=dtype)


@pytest.mark.parametrize("weight", WEIGHTS)
@pytest.mark.parametrize("gamma", [True, False])
@pytest.mark.parametrize("D", [96, 33])
def test_weights_and_intensity(weight, gamma, D):
    run_all(make(2, 300, D, F, gamma, seed=7), weight)
    run_all(make(2, 300, D, BF, gamma, seed=8, state=False), weight)


@pytest.mark.parametrize("dtype,y_dtype,grad_dtype", [(BF, F, BF), (BF, BF, F), (F, BF, BF), (F, F, BF), (F, BF, F)])
def test_types(dtype, y_dtype, grad_dtype):
    run_all(make(2, 200, 130, dtype, seed=11), osr.SCAN_NORM, y_dtype=y_dtype, grad_dtype=grad_dtype)


@pytest.mark.parametrize("mean", [-3.0, 0.0, 6.0, 9.0])
def test_strong_and_weak_forgetting(mean):
    for w in WEIGHTS:
        run_all(make(1, 700, 64, F, seed=12, mean=mean), w)


@pytest.mark.parametrize("D", [64, 65])
@pytest.mark.parametrize("dtype", [BF, F])
def test_padded_batch(D, dtype):
    """Lengths 0, 1, T, inside, at and next to the borders of tiles, and out of range; padding holds NaN,
    infinities and the types' lowest values and reaches nothing."""
    T = 400
    lens = [0, 1, T, 127, 128, 129, 256, 333, -5, T + 50]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = make(len(lens), T, D, dtype, seed=13)
    bad = [math.nan, math.inf, -math.inf, torch.finfo(dtype).min]
    for i, k in enumerate(lens):
        k = max(0, min(T, k))
        for j, name in enumerate(("v", "mu_logit", "gamma_logit")):
            x[name][i, k:] = bad[(i + j) % 4]
    clean = {k: torch.nan_to_num(t, 0.0, 0.0, 0.0) if t.dim() == 3 else t for k, t in x.items()}
    B = len(lens)
    dy, dso = grads_of(B, T, D, dtype)
    for i, k in enumerate(lens):
        dy[i, max(0, min(T, k)):] = bad[i % 4]
    for w in WEIGHTS:
        kw = dict(gamma_logit=x["gamma_logit"], lengths=n, input_weight=w)
        y, st, saved = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], y_dtype=dtype, save=True, **kw)
        g = osr.lattice_osr_scan_bwd(x["v"], x["mu_logit"], dy, dso, saved=saved, grad_dtype=dtype, **kw)
        out, bound = oracle(clean, w, n, torch.nan_to_num(dy, 0.0, 0.0, 0.0), dso)
        got = dict(g, y=y, state_out=st)
        for name in got:
            check(name, got[name], out[name], bound[name])
        for i, k in enumerate(lens):
            k = max(0, min(T, k))
            for name in ("y", "dv", "dmu_logit", "dgamma_logit"):
                assert (got[name][i, k:] == 0).all(), (name, i)
            if k == 0:
                assert torch.equal(st[i], x["state_in"][i]) and torch.equal(g["dstate_in"][i], dso[i])


def test_lengths_across_every_level():
    """Sequences that end at, before and behind the borders of runs, tiles, groups of tiles and groups of
    groups, in one batch, next to an empty one."""
    T, D = 17000, 5
    lens = [0, 1, 31, 33, 127, 129, 256, 257, 1023, 1025, 2047, 2048, 2049, 8191, 8192, 8193, 16383, 16384, 16385, T]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = make(len(lens), T, D, F, seed=18, mean=4.0)
    got = run_all(x, osr.SCAN_COMPLEMENT, n)
    for i, k in enumerate(lens):
        for name in ("y", "dv", "dmu_logit", "dgamma_logit"):
            assert (got[name][i, k:] == 0).all(), (name, i)


def test_state_in_place_at_every_length():
    """state_out is state_in: every tile that reads the old state does so before the last one writes."""
    for T in (1, 200, 257, 700, 2100, 20000):
        x = make(3, T, 70, BF, seed=T)
        want = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"])
        for _ in range(3):
            st = x["state_in"].clone()
            y, _ = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], st, gamma_logit=x["gamma_logit"], state_out=st)
            assert torch.equal(y, want[0]) and torch.equal(st, want[1]), T


def test_all_sequences_empty():
    x = make(3, 50, 40, BF)
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    got = run_all(x, osr.SCAN_ONE, n)
    assert (got["y"] == 0).all() and torch.equal(got["state_out"], x["state_in"])


@pytest.mark.parametrize("weight", WEIGHTS)
@pytest.mark.parametrize("dtype", [BF, F])
def test_documents_packed_in_a_row(weight, dtype):
    """Forget logits of -inf and of the type's lowest value drop the state, +inf and the highest keep it:
    exactly, with zero gradients; the row equals its documents one by one."""
    x = make(2, 300, 66, dtype, seed=17)
    cuts = [0, 100, 128, 129, 250]
    for c, val in zip(cuts[1:], (-math.inf, torch.finfo(dtype).min, -math.inf, -math.inf)):
        x["mu_logit"][:, c] = val
    x["mu_logit"][:, 40], x["mu_logit"][:, 200] = math.inf, torch.finfo(dtype).max
    x["state_in"][0] = 1e30
    got = run_all(x, weight, y_dtype=F)
    assert (got["dmu_logit"][:, cuts[1:] + [40, 200]] == 0).all()
    for a, b in zip(cuts, cuts[1:] + [300]):
        part = {k: t[:, a:b].contiguous() for k, t in x.items() if t.dim() == 3}
        y, _ = osr.lattice_osr_scan_fwd(part["v"], part["mu_logit"], x["state_in"] if a == 0 else None,
                                        gamma_logit=part["gamma_logit"], input_weight=weight)
        out, bound = layer.scan(part["v"], part["mu_logit"], part["gamma_logit"], x["state_in"] if a == 0 else None,
                                None, weight)
        check(f"document {a}", y, out["y"], bound["y"])
        check(f"document {a} in the row", got["y"][:, a:b], out["y"], bound["y"])


def test_nan_stays_in_its_channel_and_behind():
    x = make(2, 300, 64, F, seed=19)
    x["mu_logit"][0, 150, 7] = math.nan
    x["v"][1, 20, 9] = math.nan
    y, st = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"])
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, 150:, 7] = True
    bad[1, 20:, 9] = True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(torch.isnan(st), bad[:, -1])


def test_any_nan_passes_from_tile_to_tile():
    """A NaN of any bits (all ones is what an empty hand-off word looks like) in a logit or a value reaches the end of
    its channel, over every level of the hand-off, and no other channel."""
    T = 17000
    x = make(1, T, 64, F, seed=20, mean=3.0)
    bits = x["mu_logit"].view(torch.int32)
    bits[0, 10, 3], bits[0, 3000, 4], bits[0, 16000, 5] = -1, 0x7f800001, -1
    x["v"].view(torch.int32)[0, 500, 6] = -1
    y, st, sv = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"], save=True)
    bad = torch.zeros_like(y, dtype=torch.bool)
    for t, c in ((10, 3), (3000, 4), (16000, 5), (500, 6)):
        bad[0, t:, c] = True
    assert torch.equal(torch.isnan(y), bad)
    g = osr.lattice_osr_scan_bwd(x["v"], x["mu_logit"], torch.ones_like(y), saved=sv, gamma_logit=x["gamma_logit"])
    keep = [c for c in range(64) if c not in (3, 4, 5, 6)]
    assert all(torch.isfinite(t[..., keep]).all() for t in g.values())
    assert torch.isnan(g["dstate_in"][0, [3, 4, 5]]).all()


@pytest.mark.parametrize("off", [1, 2, 3])
def test_unaligned_buffers(off):
    """Views that start `off` elements into an allocation, every buffer of the call among them, and
    nothing written outside them."""
    B, T, D = 2, 150, 64
    x = make(B, T, D, BF, seed=23)

    def shift(t, fill=None):
        flat = torch.full((t.numel() + 16,), math.nan, dtype=t.dtype, device="cuda")
        view = flat[off:off + t.numel()].view(t.shape)
        view.copy_(t)
        return flat, view

    s = {k: shift(t)[1] for k, t in x.items()}
    ref = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"], y_dtype=BF,
                                   save=True)
    yf, y = shift(torch.zeros(B, T, D, dtype=BF, device="cuda"))
    sf, so = shift(torch.zeros(B, D, device="cuda"))
    _, _, saved = osr.lattice_osr_scan_fwd(s["v"], s["mu_logit"], s["state_in"], gamma_logit=s["gamma_logit"],
                                           y_dtype=BF, y=y, state_out=so, save=True)
    assert torch.equal(y, ref[0]) and torch.equal(so, ref[1])
    for flat, v in ((yf, y), (sf, so)):
        assert torch.isnan(flat[:off]).all() and torch.isnan(flat[off + v.numel():]).all()
    dy, dso = grads_of(B, T, D, BF)
    kw = dict(gamma_logit=x["gamma_logit"], grad_dtype=BF)
    g0 = osr.lattice_osr_scan_bwd(x["v"], x["mu_logit"], dy, dso, saved=ref[2], **kw)
    bufs = {k: shift(t) for k, t in g0.items()}
    for _, v in bufs.values():
        v.zero_()
    osr.lattice_osr_scan_bwd(s["v"], s["mu_logit"], shift(dy)[1], shift(dso)[1], saved=saved,
                             gamma_logit=s["gamma_logit"], grad_dtype=BF, grads={k: v for k, (_, v) in bufs.items()})
    for k, (flat, v) in bufs.items():
        assert torch.equal(v, g0[k]), k
        assert torch.isnan(flat[:off]).all() and torch.isnan(flat[off + v.numel():]).all(), k


def test_heads_layout_in_place_and_optional_outputs():
    B, T, H, d = 2, 140, 3, 32
    x = make(B, T, H * d, BF, seed=29)
    four = {k: t.view(B, T, H, d) if t.dim() == 3 else t.view(B, H, d) for k, t in x.items()}
    ref = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"])
    st = four["state_in"].clone()
    y, so = osr.lattice_osr_scan_fwd(four["v"], four["mu_logit"], st, gamma_logit=four["gamma_logit"], state_out=st)
    assert y.shape == (B, T, H, d) and so.data_ptr() == st.data_ptr()
    assert torch.equal(y.view(B, T, -1), ref[0]) and torch.equal(st.view(B, -1), ref[1])


@pytest.mark.parametrize("cut", [1, 64, 128, 200])
def test_split_sequence_continues(cut):
    """Two calls chained through the state, and the second part token by token, stay within the bars of one call."""
    x = make(2, 260, 66, BF, seed=31)
    out, bound = oracle(x, osr.SCAN_COMPLEMENT)
    part = lambda a, b: [x[k][:, a:b].contiguous() for k in ("v", "mu_logit", "gamma_logit")]
    v, f, g = part(0, cut)
    y1, st = osr.lattice_osr_scan_fwd(v, f, x["state_in"], gamma_logit=g)
    v, f, g = part(cut, 260)
    y2, st2 = osr.lattice_osr_scan_fwd(v, f, st, gamma_logit=g)
    check("two calls", torch.cat([y1, y2], 1), out["y"], bound["y"])
    check("state", st2, out["state_out"], bound["state_out"])
    ys, state = [], st.clone()
    for t in range(cut, 260):
        v, f, g = part(t, t + 1)
        yt, state = osr.lattice_osr_scan_step(v, f, state, gamma_logit=g, state_out=state)
        ys.append(yt.clone())
    check("steps", torch.cat([y1] + ys, 1), out["y"], bound["y"])
    check("state after steps", state, out["state_out"], bound["state_out"])


@pytest.mark.parametrize("B,D", [(1, 1), (1, 64), (3, 33), (300, 130), (17, 4096)])
@pytest.mark.parametrize("dtype,y_dtype", [(BF, BF), (BF, F), (F, F)])
def test_step(B, D, dtype, y_dtype):
    for w in WEIGHTS:
        for gamma in (True, False):
            x = make(B, 1, D, dtype, gamma, seed=37)
            y, st = osr.lattice_osr_scan_step(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"],
                                              input_weight=w, y_dtype=y_dtype)
            out, bound = oracle(x, w)
            check("y", y, out["y"], bound["y"])
            check("state", st, out["state_out"], bound["state_out"])


@pytest.mark.parametrize("B,T,D", [(1, 20000, 130), (2, 4100, 2048), (9, 1100, 512)])
def test_long_and_wide(B, T, D):
    """Few channels over many tiles, and enough sequences to fill the chip."""
    run_all(make(B, T, D, BF, seed=41, mean=3.0), osr.SCAN_NORM, y_dtype=BF, grad_dtype=BF)


def test_reruns_agree_bit_for_bit():
    x = make(2, 9000, 384, BF, seed=43)
    dy, dso = grads_of(2, 9000, 384, BF)
    first = None
    for _ in range(4):
        y, st, sv = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"],
                                             save=True)
        g = osr.lattice_osr_scan_bwd(x["v"], x["mu_logit"], dy, dso, saved=sv, gamma_logit=x["gamma_logit"])
        got = [y, st, *g.values()]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_workspace_contents_do_not_matter():
    """Whatever the workspace and `saved` hold on entry, hand-off words that look filled among it; nothing is
    written behind either."""
    B, T, D = 2, 20000, 130
    x = make(B, T, D, BF, seed=47, mean=3.0)
    dy, dso = grads_of(B, T, D, BF)
    desc = osr.make_scan_desc(B, T, D, osr.BF16, osr.BF16, osr.F32)
    wn, sn = osr.lattice_osr_scan_workspace_bytes(desc), osr.lattice_osr_scan_saved_bytes(desc)
    first = None
    for fill in (0, 255, 0x3f, 0x7f, None):
        ws, sv = (torch.empty(n + 256, dtype=torch.uint8, device="cuda") for n in (wn, sn))
        for t in (ws, sv):
            t.random_(0, 256) if fill is None else t.fill_(fill)
        tails = [ws[wn:].clone(), sv[sn:].clone()]
        y, st, _ = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"],
                                            y_dtype=BF, saved=sv[:sn], workspace=ws[:wn])
        g = osr.lattice_osr_scan_bwd(x["v"], x["mu_logit"], dy, dso, saved=sv[:sn], gamma_logit=x["gamma_logit"],
                                     workspace=ws[:wn])
        got = [y, st, *g.values()]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got)), fill
        assert torch.equal(ws[wn:], tails[0]) and torch.equal(sv[sn:], tails[1]), fill


def test_two_streams_at_once():
    """Calls on two streams, each with its own buffers, and a call under another stream than the current."""
    xs = [make(2, 6000, 256, BF, seed=50 + i) for i in range(2)]
    want = [osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"]) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for _ in range(3):
        got = [osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"], stream=s)
               for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


def test_captured_and_replayed():
    """Forward, backward and step in one graph, replayed with new inputs between eager work; the workspace is
    shared by the graph's own calls and by a second graph."""
    B, T, D = 2, 3000, 256
    x = make(B, T, D, BF, seed=61)
    dy, dso = grads_of(B, T, D, BF)
    desc = osr.make_scan_desc(B, T, D, osr.BF16, osr.BF16, osr.BF16)
    ws = torch.empty(max(16, osr.lattice_osr_scan_workspace_bytes(desc)), dtype=torch.uint8, device="cuda")

    def step(tag):
        y, st, sv = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"],
                                             y_dtype=BF, save=True, workspace=ws)
        g = osr.lattice_osr_scan_bwd(x["v"], x["mu_logit"], dy, dso, saved=sv, gamma_logit=x["gamma_logit"],
                                     grad_dtype=BF, workspace=ws)
        t = [x[k][:, :1].contiguous() for k in ("v", "mu_logit", "gamma_logit")]
        ys, ss = osr.lattice_osr_scan_step(t[0], t[1], st, gamma_logit=t[2])
        return [y, st, *g.values(), ys, ss]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step("warm")
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step("capture"))
        graphs.append(g)
    for i in range(4):
        new = make(B, T, D, BF, seed=70 + i)
        for k in x:
            x[k].copy_(new[k])
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs[i % 2]]
        want = step("eager")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), i


def test_offsets_past_32_bits():
    """A batch whose tensors hold more than 2^32 bytes and 2^31 elements: its last sequence equals a call of its own."""
    B, T, D = 9, 65536, 4096
    v = torch.randn((1, T, D), device="cuda").to(BF)
    f = (torch.randn((1, T, D), device="cuda") + 2).to(BF)
    want = osr.lattice_osr_scan_fwd(v, f, None, y_dtype=BF, save=True)
    dy = torch.randn((1, T, D), device="cuda").to(BF)
    gw = osr.lattice_osr_scan_bwd(v, f, dy, saved=want[2], grad_dtype=BF)
    big = [torch.zeros((B, T, D), dtype=BF, device="cuda") for _ in range(3)]
    for b, t in zip(big, (v, f, dy)):
        b[-1] = t[0]
    got = osr.lattice_osr_scan_fwd(big[0], big[1], None, y_dtype=BF, save=True)
    assert torch.equal(got[0][-1], want[0][0]) and torch.equal(got[1][-1], want[1][0])
    assert (got[0][:-1] == 0).all()
    g = osr.lattice_osr_scan_bwd(big[0], big[1], big[2], saved=got[2], grad_dtype=BF)
    for k in ("dv", "dmu_logit", "dstate_in"):
        assert torch.equal(g[k][-1], gw[k][0]), k
        assert (g[k][:-1] == 0).all()


def test_widest_rows():
    """The most channels a call takes: a tile's rows reach the largest offsets; any 64 of them equal a call of
    their own."""
    T, D = 270, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(90)
    v = torch.randn((1, T, D), generator=g, device="cuda")
    f = torch.randn((1, T, D), generator=g, device="cuda") + 2
    y, st, sv = osr.lattice_osr_scan_fwd(v, f, save=True)
    gr = osr.lattice_osr_scan_bwd(v, f, y, saved=sv)
    for c in (0, 12345 * 64, D - 64):
        part = [t[..., c:c + 64].contiguous() for t in (v, f, y)]
        y2, st2, sv2 = osr.lattice_osr_scan_fwd(part[0], part[1], save=True)
        g2 = osr.lattice_osr_scan_bwd(part[0], part[1], part[2], saved=sv2)
        assert torch.equal(y[..., c:c + 64], y2) and torch.equal(st[..., c:c + 64], st2)
        for k in ("dv", "dmu_logit", "dstate_in"):
            assert torch.equal(gr[k][..., c:c + 64], g2[k]), k
    with pytest.raises(osr.OSRError):
        osr.lattice_osr_scan_fwd(*[torch.zeros((1, 1, D + 1), dtype=BF, device="cuda")] * 2)


def test_empty_batch_is_refused():
    for shape in ((0, 4, 8), (2, 0, 8), (2, 4, 0)):
        t = torch.zeros(shape, dtype=BF, device="cuda")
        with pytest.raises(osr.OSRError) as e:
            osr.lattice_osr_scan_fwd(t, t)
        assert e.value.status == osr.ERR_SHAPE


def test_infinite_values_follow_the_formula():
    """An infinite input makes its channel infinite until a gate of 0 meets it (0 times infinity: NaN), and no other."""
    x = make(1, 600, 64, F, seed=91, gamma=False)
    x["v"][0, 100, 3] = math.inf
    x["mu_logit"][0, 400, 3] = -math.inf
    y, _ = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], input_weight=osr.SCAN_ONE)
    assert torch.isfinite(y[0, :100]).all() and torch.isinf(y[0, 100:400, 3]).all() and torch.isnan(y[0, 400:, 3]).all()
    keep = torch.arange(64, device="cuda") != 3
    assert torch.isfinite(y[..., keep]).all()


def test_longest_sequences():
    """One channel past 2^28 tokens, more than half of the tiles that a call takes: what follows a dropped state
    equals a call of its own, and so does the beginning."""
    p, T = 1 << 28, (1 << 28) + 3 * 16384 + 777
    g = torch.Generator(device="cuda").manual_seed(92)
    v, f, dy = (torch.randn((1, T, 1), generator=g, device="cuda", dtype=BF) for _ in range(3))
    f += 2
    f[0, p] = -math.inf
    y, st, sv = osr.lattice_osr_scan_fwd(v, f, y_dtype=BF, save=True)
    gr = osr.lattice_osr_scan_bwd(v, f, dy, saved=sv, grad_dtype=BF)
    assert all(torch.isfinite(t).all() for t in (y, *gr.values()))
    head = [t[:, :16384].contiguous() for t in (v, f)]
    assert torch.equal(y[:, :16384], osr.lattice_osr_scan_fwd(*head, y_dtype=BF)[0])
    part = [t[:, p:].contiguous() for t in (v, f, dy)]
    y2, st2, sv2 = osr.lattice_osr_scan_fwd(part[0], part[1], y_dtype=BF, save=True)
    g2 = osr.lattice_osr_scan_bwd(*part, saved=sv2, grad_dtype=BF)
    assert torch.equal(y[:, p:], y2) and torch.equal(st, st2)
    for k in ("dv", "dmu_logit"):
        assert torch.equal(gr[k][:, p:], g2[k]), k


@pytest.mark.parametrize("call", ["step", "forward"])
def test_gates_alone(call):
    """mu, 1 - mu and gamma by themselves (y = mu 1 + 0, (1 - mu) 1 and gamma 1), logits from -80 to 80: fp32 within
    8 units of 2^-24 of each gate's own value (2^x 2, its low part 1, 1 + e 1, 1 / x 2, e s 1, and 1 for what is of
    second order); bf16 logits, whose exponent is one rounded product, within 8 and 1.25 |x| more."""
    x = torch.cat([torch.linspace(-80, 80, 20001), torch.linspace(-3, 3, 3000)]).cuda().view(1, 1, -1)
    for dtype in (F, BF):
        f = x.to(dtype)
        one, zero = torch.ones_like(f), torch.zeros_like(f)
        st = torch.ones((1, f.shape[-1]), device="cuda")
        run = osr.lattice_osr_scan_step if call == "step" else osr.lattice_osr_scan_fwd
        mu, _ = run(zero, f, st)
        om, _ = run(one, f, 0 * st)
        gam, _ = run(one, zero, 0 * st, gamma_logit=f, input_weight=osr.SCAN_ONE)
        lim = 8 * layer.U * (1 if dtype == F else 1 + 1.25 / 8 * f.double().abs())
        for name, got, ref in (("mu", mu, torch.sigmoid(f.double())), ("1 - mu", om, torch.sigmoid(-f.double())),
                               ("gamma", gam, torch.sigmoid(f.double()))):
            worst = float(((got.double() / ref - 1).abs() / lim).max())
            print(f"  {dtype} {name}: {worst:.3f}", flush=True)
            assert worst <= 1, (dtype, name, worst)


def test_refusals_carry_the_library_s_status():
    """A descriptor that a call refuses is reported as the C ABI reports it, also where its sizes are asked first."""
    x = make(2, 200, 40, BF)
    y, _, saved = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], save=True)
    for bad in (-1, 3):
        for call in (lambda: osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], input_weight=bad),
                     lambda: osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], input_weight=bad, save=True),
                     lambda: osr.lattice_osr_scan_bwd(x["v"], x["mu_logit"], y, saved=saved, input_weight=bad)):
            with pytest.raises(osr.OSRError) as e:
                call()
            assert e.value.status == osr.ERR_UNSUPPORTED


@pytest.mark.parametrize("T", [33, 300, 3000, 20000])
@pytest.mark.parametrize("dtype", [F, BF])
def test_infinite_states_stay_infinite_under_strong_forgetting(T, dtype):
    """Gates whose product over a run underflows, none of them 0: an infinite state, input or incoming gradient is
    infinite from there on, as token by token, at every level of the split; a gate of 0 still drops a finite one."""
    x = make(1, T, 64, dtype, seed=93, mean=-4.0)
    x["state_in"][0, 3], x["state_in"][0, 5] = math.inf, -math.inf
    x["v"][0, T // 3, 7] = math.inf
    x["mu_logit"][0, T // 2, 9] = -math.inf
    for w in WEIGHTS:
        y, st, sv = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"],
                                             input_weight=w, save=True)
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[0, :, [3, 5]] = True
        bad[0, T // 3:, 7] = True
        assert torch.equal(torch.isinf(y), bad) and not torch.isnan(y).any()
        assert torch.equal(torch.isinf(st), bad[:, -1])
        assert (y[0, :, 3] > 0).all() and (y[0, :, 5] < 0).all()
        clean = {k: torch.nan_to_num(t, 0.0, 0.0, 0.0) if k in ("v", "state_in") else t for k, t in x.items()}
        _, _, sv = osr.lattice_osr_scan_fwd(clean["v"], x["mu_logit"], clean["state_in"],
                                            gamma_logit=x["gamma_logit"], input_weight=w, save=True)
        dy, dso = grads_of(1, T, 64, F)
        dso[0, 3], dso[0, 5] = math.inf, -math.inf
        dy[0, T // 3, 7] = math.inf
        g = osr.lattice_osr_scan_bwd(clean["v"], x["mu_logit"], dy, dso, saved=sv, gamma_logit=x["gamma_logit"],
                                     input_weight=w)
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[0, :, [3, 5]] = True
        bad[0, :T // 3 + 1, 7] = True
        assert torch.equal(torch.isinf(g["dv"]), bad) and not torch.isnan(g["dv"]).any()
        assert torch.equal(torch.isinf(g["dstate_in"]), bad[:, 0])
        assert (g["dv"][0, :, 3] > 0).all() and (g["dv"][0, :, 5] < 0).all()


@pytest.mark.parametrize("T", [1, 100, 700])
def test_outputs_that_are_not_wanted(T):
    """The C calls without state_out, saved, dstate_in: the rest bit for bit, whatever is left out."""
    import ctypes

    B, D = 3, 70
    x = make(B, T, D, F, seed=94)
    desc = osr.make_scan_desc(B, T, D, osr.F32, osr.F32, osr.F32)
    lib, ref, ptr = osr.load_library(), ctypes.byref(desc), lambda t: None if t is None else t.data_ptr()
    st = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(max(16, osr.lattice_osr_scan_workspace_bytes(desc)), dtype=torch.uint8, device="cuda")
    y, so, sv = osr.lattice_osr_scan_fwd(x["v"], x["mu_logit"], x["state_in"], gamma_logit=x["gamma_logit"], save=True)
    dy, dso = grads_of(B, T, D, F)
    g = osr.lattice_osr_scan_bwd(x["v"], x["mu_logit"], dy, dso, saved=sv, gamma_logit=x["gamma_logit"])
    for saved in (None, torch.zeros_like(sv)):
        y2 = torch.empty_like(y)
        assert lib.lattice_osr_scan_fwd(ref, ptr(x["v"]), ptr(x["mu_logit"]), ptr(x["gamma_logit"]), None,
                                        ptr(x["state_in"]), None, ptr(y2), ptr(saved), sv.numel() if saved is not None
                                        else 0, ptr(ws), ws.numel(), st) == osr.OK
        assert torch.equal(y, y2) and (saved is None or torch.equal(saved, sv))
    outs = [torch.empty_like(y) for _ in range(3)]
    assert lib.lattice_osr_scan_bwd(ref, ptr(x["v"]), ptr(x["mu_logit"]), ptr(x["gamma_logit"]), None, ptr(sv),
                                    sv.numel(), ptr(dy), ptr(dso), *[ptr(t) for t in outs], None, ptr(ws), ws.numel(),
                                    st) == osr.OK
    assert all(torch.equal(a, g[k]) for a, k in zip(outs, ("dv", "dmu_logit", "dgamma_logit")))
