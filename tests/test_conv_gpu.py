"""GPU parity of the short causal convolution (lattice_osr_conv_*) against the
fp64 oracle (oracle/mixer.py), element by element, at the oracle's own bounds
plus half a step of a bf16 output."""
import math

import pytest
import torch

from compressed_memory_linear_amd import osr
from oracle import mixer

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def make(B, T, D, W=4, dtype=BF, seed=0, bias=True, hist=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    return dict(x=r(B, T, D).to(dtype), w=0.5 * r(D, W), bias=r(D) if bias else None,
                hist_in=r(B, W - 1, D).to(dtype) if hist else None)


def check(name, got, ref, bound):
    ref, bound = ref.reshape(got.shape), bound.reshape(got.shape)
    err = (got.double() - ref).abs()
    some = torch.isfinite(bound)  # where the oracle has one
    assert torch.isfinite(got[some]).all(), name
    worst = float((err / mixer.rounded(bound, ref, got.dtype))[some].max()) if some.any() else 0.0
    print(f"  {name}: worst error / bar {worst:.3f}", flush=True)
    assert worst <= 1.0, (name, worst)


def run_all(x, act=osr.CONV_SILU, y_dtype=F, grad_dtype=F, seed=0, lengths=None, segments=None, oracle_x=None,
            spoil=None):
    B, T, D = x["x"].shape
    W = x["w"].shape[1]
    print(f"conv B{B} T{T} D{D} W{W} {x['x'].dtype} y {y_dtype} grad {grad_dtype} act {act} lengths "
          f"{lengths is not None} segments {segments is not None}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    dy = torch.randn((B, T, D), generator=g, device="cuda").to(y_dtype)
    dho = torch.randn((B, W - 1, D), generator=g, device="cuda").to(grad_dtype)
    kw = dict(act=act, lengths=lengths, segments=segments)
    y, ho = osr.lattice_osr_conv_fwd(x["x"], x["w"], x["bias"], x["hist_in"], y_dtype=y_dtype, return_history=True, **kw)
    clean = dy
    if spoil is not None:
        dy = spoil(dy)
    got = osr.lattice_osr_conv_bwd(x["x"], x["w"], dy, x["bias"], x["hist_in"], dho, grad_dtype=grad_dtype, **kw)
    torch.cuda.synchronize()
    got = dict(got, y=y, hist_out=ho)
    out, bound = mixer.conv(**(oracle_x or x), **kw, dy=clean, dhist_out=dho)
    for n in got:
        if got[n].numel():
            check(n, got[n], out[n], bound[n])
    return got


SHAPES = [(1, 1, 1), (2, 3, 5), (1, 16, 64), (3, 17, 66), (2, 128, 40), (2, 129, 130), (1, 1000, 257), (40, 9, 24),
          (2, 511, 1000)]


@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F])
def test_shapes(B, T, D, dtype):
    run_all(make(B, T, D, dtype=dtype, seed=T), y_dtype=dtype, grad_dtype=dtype)


@pytest.mark.parametrize("W", range(1, 9))
@pytest.mark.parametrize("act", [osr.CONV_NONE, osr.CONV_SILU])
@pytest.mark.parametrize("D", [40, 33])
def test_widths(W, act, D):
    run_all(make(2, 150, D, W, F, seed=W, bias=W % 2 == 0, hist=W % 3 != 0), act)
    run_all(make(2, 3, D, W, BF, seed=W), act, y_dtype=BF, grad_dtype=BF)  # fewer tokens than taps


@pytest.mark.parametrize("dtype,y_dtype,grad_dtype", [(BF, F, BF), (BF, BF, F), (F, BF, BF), (F, F, BF), (F, BF, F)])
def test_types(dtype, y_dtype, grad_dtype):
    run_all(make(2, 140, 72, dtype=dtype, seed=4), y_dtype=y_dtype, grad_dtype=grad_dtype)


@pytest.mark.parametrize("W", [2, 4, 7])
@pytest.mark.parametrize("D", [64, 65])
@pytest.mark.parametrize("dtype", [BF, F])
def test_padded_batch(W, D, dtype):
    """Lengths 0, 1, T, shorter than the filter, at and next to the borders of runs, and out of range; padding
    holds NaN, infinities and the types' lowest values and reaches nothing."""
    T = 300
    lens = [0, 1, 2, 3, T, 15, 16, 17, 127, 128, 129, 130, 131, 257, -5, T + 50]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = make(len(lens), T, D, W, dtype, seed=13)
    clean = dict(x, x=x["x"].clone())
    bad = [math.nan, math.inf, -math.inf, torch.finfo(dtype).min]
    for i, k in enumerate(lens):
        k = max(0, min(T, k))
        x["x"][i, k:] = bad[i % 4]
        clean["x"][i, k:] = 0

    def spoil(dy):
        dy = dy.clone()
        for i, k in enumerate(lens):
            dy[i, max(0, min(T, k)):] = bad[(i + 1) % 4]
        return dy

    got = run_all(x, y_dtype=dtype, grad_dtype=dtype, lengths=n, oracle_x=clean, spoil=spoil)
    for i, k in enumerate(lens):
        k = max(0, min(T, k))
        assert (got["y"][i, k:] == 0).all() and (got["dx"][i, k:] == 0).all(), i
        if k == 0:
            assert torch.equal(got["hist_out"][i], x["hist_in"][i])


@pytest.mark.parametrize("W", [2, 4, 8])
@pytest.mark.parametrize("dtype", [BF, F])
def test_documents_packed_in_a_row(W, dtype):
    """Borders at, before and behind those of runs, one and two tokens apart, at the very end, in padding, and
    numbers that come again; the row equals its documents one by one, exactly, and hist_out continues it."""
    T = 300
    cuts = [0, 2, 15, 16, 17, 32, 127, 128, 129, 131, 200, 298]
    seg = torch.zeros((3, T), dtype=torch.int32, device="cuda")
    for i, c in enumerate(cuts):
        seg[:, c:] = [7, 3, 7, -1, 2 ** 31 - 1][i % 5]
    n = torch.tensor([T, 130, 299], dtype=torch.int32, device="cuda")
    x = make(3, T, 40, W, dtype, seed=17)
    x["x"][:, 50] = torch.finfo(dtype).max / 4  # a large value stays in its document
    got = run_all(x, y_dtype=dtype, grad_dtype=F, lengths=n, segments=seg)
    for a, b in zip(cuts, cuts[1:] + [T]):
        y, ho = osr.lattice_osr_conv_fwd(x["x"][:1, a:b].contiguous(), x["w"], x["bias"],
                                         x["hist_in"][:1] if a == 0 else None, y_dtype=dtype, return_history=True)
        assert torch.equal(y, got["y"][:1, a:b]), a
    assert torch.equal(ho, got["hist_out"][:1])


def test_a_border_stops_what_is_not_finite():
    x = make(1, 60, 8, 4, F, seed=18)
    seg = (torch.arange(60, device="cuda") >= 30).int().view(1, 60)
    want = osr.lattice_osr_conv_fwd(x["x"], x["w"], x["bias"], x["hist_in"], segments=seg)
    x["x"][0, 29] = math.nan
    got = osr.lattice_osr_conv_fwd(x["x"], x["w"], x["bias"], x["hist_in"], segments=seg)
    assert torch.equal(got[:, 30:], want[:, 30:]) and torch.isnan(got[:, 29]).all()
    dy = torch.ones_like(x["x"])
    dy[0, 30] = math.nan
    g = osr.lattice_osr_conv_bwd(x["x"], x["w"], dy, x["bias"], x["hist_in"], segments=seg)
    assert torch.isfinite(g["dx"][:, :26]).all() and torch.isnan(g["dx"][:, 30]).all()
    assert torch.isnan(g["dx"][:, 26:30]).all()  # from the NaN in token 29's own sum


def shifted(t, off):
    flat = torch.full((t.numel() + 16,), math.nan, dtype=t.dtype, device="cuda")
    view = flat[off:off + t.numel()].view(t.shape)
    view.copy_(t)
    return flat, view


@pytest.mark.parametrize("off", [1, 2, 3])
def test_unaligned_buffers(off):
    B, T, D = 2, 150, 64
    x = make(B, T, D, seed=23)
    s = {k: shifted(t, off)[1] for k, t in x.items()}
    ref = osr.lattice_osr_conv_fwd(x["x"], x["w"], x["bias"], x["hist_in"], return_history=True)
    outs = [shifted(torch.zeros_like(t), off) for t in ref]
    osr.lattice_osr_conv_fwd(s["x"], s["w"], s["bias"], s["hist_in"], y=outs[0][1], hist_out=outs[1][1])
    dy, dho = torch.randn(B, T, D, device="cuda").to(BF), torch.randn(B, 3, D, device="cuda").to(BF)
    g0 = osr.lattice_osr_conv_bwd(x["x"], x["w"], dy, x["bias"], x["hist_in"], dho, grad_dtype=BF)
    bufs = {k: shifted(torch.zeros_like(t), off) for k, t in g0.items()}
    osr.lattice_osr_conv_bwd(s["x"], s["w"], shifted(dy, off)[1], s["bias"], s["hist_in"], shifted(dho, off)[1],
                             grad_dtype=BF, grads={k: v for k, (_, v) in bufs.items()})
    for (flat, v), want in zip(outs + list(bufs.values()), list(ref) + list(g0.values())):
        # the same sums in the same order, but for how many channels a thread has
        torch.testing.assert_close(v, want, rtol=0, atol=0)
        assert torch.isnan(flat[:off]).all() and torch.isnan(flat[off + v.numel():]).all()


@pytest.mark.parametrize("D", [64, 66, 3])
def test_rows_a_stride_apart(D):
    """x as one half of a projection's output, its other half NaN."""
    x = make(2, 70, D, seed=25)
    wide = torch.full((2, 70, 2 * D), math.nan, dtype=BF, device="cuda")
    for at in (0, D):
        v = wide[..., at:at + D]
        v.copy_(x["x"])
        dy = torch.randn(2, 70, D, device="cuda").to(BF)
        n = torch.tensor([70, 33], dtype=torch.int32, device="cuda")
        kw = dict(lengths=n)
        a = osr.lattice_osr_conv_fwd(x["x"], x["w"], x["bias"], x["hist_in"], return_history=True, **kw)
        b = osr.lattice_osr_conv_fwd(v, x["w"], x["bias"], x["hist_in"], return_history=True, **kw)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        ga = osr.lattice_osr_conv_bwd(x["x"], x["w"], dy, x["bias"], x["hist_in"], **kw)
        gb = osr.lattice_osr_conv_bwd(v, x["w"], dy, x["bias"], x["hist_in"], **kw)
        assert all(torch.equal(ga[k], gb[k]) for k in ga)
        one = osr.lattice_osr_conv_step(v[:, 5:6], x["w"], x["hist_in"], x["bias"])
        two = osr.lattice_osr_conv_step(x["x"][:, 5:6].contiguous(), x["w"], x["hist_in"], x["bias"])
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
        wide.fill_(math.nan)


@pytest.mark.parametrize("W", [2, 4, 8])
@pytest.mark.parametrize("D", [64, 33])
def test_split_sequence_and_single_tokens(W, D):
    """Calls chained through the history, of any length, and single tokens: exactly the one call's outputs."""
    x = make(2, 100, D, W, seed=31)
    y, ho = osr.lattice_osr_conv_fwd(x["x"], x["w"], x["bias"], x["hist_in"], return_history=True)
    ys, h, at = [], x["hist_in"], 0
    for n in (1, 2, 3, 16, 40, 38):
        yt, h = osr.lattice_osr_conv_fwd(x["x"][:, at:at + n].contiguous(), x["w"], x["bias"], h, return_history=True)
        ys.append(yt)
        at += n
    assert torch.equal(torch.cat(ys, 1), y) and torch.equal(h, ho)
    ys, h = [], x["hist_in"].clone()
    for t in range(100):
        yt, _ = osr.lattice_osr_conv_step(x["x"][:, t:t + 1].contiguous(), x["w"], h, x["bias"], hist_out=h)
        ys.append(yt)
    assert torch.equal(torch.cat(ys, 1), y) and torch.equal(h, ho)


@pytest.mark.parametrize("B,D,W", [(1, 1, 2), (1, 2048, 4), (3, 33, 3), (300, 130, 4), (17, 4096, 8)])
@pytest.mark.parametrize("dtype,y_dtype", [(BF, BF), (BF, F), (F, F)])
def test_step(B, D, W, dtype, y_dtype):
    for act in (osr.CONV_NONE, osr.CONV_SILU):
        x = make(B, 1, D, W, dtype, seed=37, bias=act == osr.CONV_SILU)
        y, ho = osr.lattice_osr_conv_step(x["x"], x["w"], x["hist_in"], x["bias"], act=act, y_dtype=y_dtype)
        out, bound = mixer.conv(**x, act=act)
        check("y", y, out["y"], bound["y"])
        assert torch.equal(ho.double(), out["hist_out"])


def test_heads_layout_reruns_and_capture():
    B, T, H, d, W = 2, 140, 3, 32, 4
    x = make(B, T, H * d, W, seed=41)
    dy = torch.randn(B, T, H * d, device="cuda").to(BF)
    y = osr.lattice_osr_conv_fwd(x["x"], x["w"], x["bias"], x["hist_in"])
    g = osr.lattice_osr_conv_bwd(x["x"], x["w"], dy, x["bias"], x["hist_in"])
    four = dict(x=x["x"].view(B, T, H, d), w=x["w"].view(H, d, W), bias=x["bias"].view(H, d),
                hist_in=x["hist_in"].view(B, W - 1, H, d))
    assert torch.equal(osr.lattice_osr_conv_fwd(**four).view_as(y), y)
    g4 = osr.lattice_osr_conv_bwd(four["x"], four["w"], dy.view(B, T, H, d), four["bias"], four["hist_in"])
    for k in g:
        assert torch.equal(g4[k].reshape(g[k].shape), g[k]), k
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        osr.lattice_osr_conv_bwd(x["x"], x["w"], dy, x["bias"], x["hist_in"])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg = osr.lattice_osr_conv_fwd(x["x"], x["w"], x["bias"], x["hist_in"])
        gg = osr.lattice_osr_conv_bwd(x["x"], x["w"], dy, x["bias"], x["hist_in"])
    for _ in range(3):
        yg.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, y) and all(torch.equal(gg[k], g[k]) for k in g)
        osr.lattice_osr_conv_fwd(x["x"], x["w"])
        torch.cuda.synchronize()
    ys = osr.lattice_osr_conv_fwd(x["x"], x["w"], x["bias"], x["hist_in"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(ys, y)


@pytest.mark.parametrize("B,T,D", [(1, 20000, 72), (2, 4100, 2048)])
def test_long_and_wide(B, T, D):
    g = torch.Generator(device="cuda").manual_seed(3)
    seg = (torch.rand((B, T), generator=g, device="cuda") < 20 / T).cumsum(1).int()
    run_all(make(B, T, D, seed=43), y_dtype=BF, grad_dtype=BF, segments=seg)


def test_most_runs_of_the_backward():
    """One run of 64 threads less than a launch of 2^32 has.  Whole numbers of unit size, so that every sum is exact
    (a thread adds 2^21 of them): dx is the filter's last tap times dy, dw and dbias are counts."""
    B = (1 << 26) - 1
    g = torch.Generator(device="cuda").manual_seed(71)
    r = lambda: torch.randint(-1, 2, (B, 1, 1), generator=g, device="cuda", dtype=torch.int8).to(BF)
    x, dy, hist = r(), r(), r()
    w, bias = torch.tensor([[2.0, -3.0]], device="cuda"), torch.ones(1, device="cuda")
    got = osr.lattice_osr_conv_bwd(x, w, dy, bias, hist, act=osr.CONV_NONE, grad_dtype=BF)
    assert torch.equal(got["dx"], -3 * dy) and torch.equal(got["dhist_in"], 2 * dy)
    count = lambda t: int(t.sum(dtype=torch.float64))
    assert got["dw"].tolist() == [[count(dy * hist), count(dy * x)]] and got["dbias"].tolist() == [count(dy)]


def test_widest_launch_of_the_forward():
    """65 channels take two waves to a run, the most lanes that idle: a launch of nearly 2^32 threads.  Whole numbers
    of up to 17, exact in bf16."""
    D = 65
    B = ((1 << 31) - 1) // D
    g = torch.Generator(device="cuda").manual_seed(73)
    x = torch.randint(-8, 9, (B, 1, D), generator=g, device="cuda", dtype=torch.int8).to(BF)
    w = torch.ones((D, 1), device="cuda") * 2
    y = osr.lattice_osr_conv_fwd(x, w, torch.full((D,), 1.0, device="cuda"), act=osr.CONV_NONE)
    assert torch.equal(y, 2 * x + 1)
