"""GPU parity of the norms around a block (lattice_osr_norm_*) against the fp64
oracle (oracle/layer.py), element by element, at the oracle's own bounds plus
half a step of a bf16 output; and the scan and the norms run together as a
layer's forward and backward.
"""
import math

import pytest
import torch

from compressed_memory_linear_amd import osr
from oracle import layer

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def make(R, D, in_dtype=BF, res_dtype=BF, gate="gelu", post=True, x=True, scale=True, pre=True, y=True, weights=True,
         seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, m=0.0, k=1.0: torch.randn(s, generator=g, device="cuda") * k + m
    t = dict(y=r(R, D).to(in_dtype), x=r(R, D, k=2.0).to(res_dtype) if x else None,
             gate=r(R, D, k=1.5).to(in_dtype) if gate else None, w_post=r(D, m=1, k=0.2) if post and weights else None,
             scale=r(D, m=0.3, k=0.1) if scale else None, w_pre=r(D, m=1, k=0.2) if pre and weights else None)
    if not y:
        t.update(y=None, gate=None, w_post=None, scale=None)
    o = dict(gate_kind={"gelu": osr.GATE_GELU, "silu": osr.GATE_SILU, None: osr.GATE_NONE}[gate if y else None],
             post_norm=post and y, pre_norm=pre, eps=1e-6)
    dx_out = r(R, D).to(res_dtype)
    dz = r(R, D).to(in_dtype) if pre else None
    return t, o, dx_out, dz


def check(name, got, ref, bound):
    err = (got.double() - ref).abs()
    lim = layer.rounded(bound, ref, got.dtype)
    assert torch.isfinite(got).all(), name
    worst = float((err / lim).max())
    print(f"  {name}: worst error / bar {worst:.3f}", flush=True)
    assert worst <= 1.0, (name, worst)


def oracle(t, o, dx_out=None, dz=None, backward=False):
    return layer.norm(**t, gate_kind=o["gate_kind"], post=o["post_norm"], pre=o["pre_norm"], eps=o["eps"],
                      dx_out=dx_out, dz=dz, backward=backward)


def run_all(t, o, dx_out, dz, grad_dtype=F, res_dtype=BF):
    lead = t["y"] if t["y"] is not None else t["x"]
    print(f"norm {tuple(lead.shape)} {lead.dtype} {o} has {[k for k, v in t.items() if v is not None]}", flush=True)
    x_out, z = osr.lattice_osr_norm_fwd(**t, **o, x_dtype=res_dtype, z_dtype=lead.dtype)
    g = osr.lattice_osr_norm_bwd(**t, **o, dx_out=dx_out, dz=dz, grad_dtype=grad_dtype)
    torch.cuda.synchronize()
    out, bound = oracle(t, o, dx_out, dz, True)
    got = dict(g)
    if x_out is not None:
        got["x_out"] = x_out
    if z is not None:
        got["z"] = z
    wants = {"d" + k for k, v in t.items() if v is not None}
    assert set(got) == wants | ({"x_out"} if t["y"] is not None else set()) | ({"z"} if o["pre_norm"] else set())
    for n in got:
        check(n, got[n], out[n], bound[n])
    return got


DIMS = [1, 2, 7, 8, 33, 64, 65, 128, 200, 256, 504, 512, 777, 1000, 1024, 1536, 2048, 2050, 4096, 5000, 8192, 8200,
        12345, 16384]


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("dtype", [BF, F])
def test_row_widths(D, dtype):
    run_all(*make(37, D, dtype, dtype, seed=D), grad_dtype=dtype, res_dtype=dtype)


@pytest.mark.parametrize("R", [1, 2, 31, 32, 33, 255, 5000])
@pytest.mark.parametrize("D", [64, 61, 1024])
def test_row_counts(R, D):
    run_all(*make(R, D, seed=R), grad_dtype=BF)


@pytest.mark.parametrize("gate", ["gelu", "silu", None])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("x", [True, False])
@pytest.mark.parametrize("pre", [True, False])
def test_combinations(gate, post, x, pre):
    for D in (96, 300):
        for scale in (True, False):
            run_all(*make(50, D, F, F, gate, post, x, scale, pre, seed=3), res_dtype=F)


@pytest.mark.parametrize("in_dtype,res_dtype,grad_dtype", [(BF, F, BF), (BF, F, F), (F, BF, F), (F, BF, BF),
                                                           (BF, BF, F), (F, F, BF)])
def test_types(in_dtype, res_dtype, grad_dtype):
    for D in (256, 1001):
        run_all(*make(70, D, in_dtype, res_dtype, seed=5), grad_dtype=grad_dtype, res_dtype=res_dtype)


def test_first_block_and_no_weights():
    """y None: the norm alone; weights None: ones."""
    run_all(*make(20, 192, BF, BF, y=False, seed=6))
    run_all(*make(20, 192, F, F, y=False, seed=6, weights=False), res_dtype=F)
    run_all(*make(20, 192, BF, F, weights=False, scale=False, seed=7), res_dtype=F)


def test_without_incoming_residual_gradient():
    t, o, _, dz = make(20, 320, BF, BF, seed=8)
    g = osr.lattice_osr_norm_bwd(**t, **o, dx_out=None, dz=dz)
    out, bound = oracle(t, o, None, dz, True)
    for n in g:
        check(n, g[n], out[n], bound[n])


def test_rows_of_zeros_and_tails_of_the_gate():
    """Empty rows (padding) stay finite: z and the gradients are those of a zero row; gates far out."""
    t, o, dx_out, dz = make(12, 64, F, F, seed=9)
    t["y"][3] = 0
    t["x"][3] = 0
    t["y"][5] = 0
    t["gate"][6] = torch.linspace(-12, 12, 64, device="cuda")
    got = run_all(t, o, dx_out, dz, res_dtype=F)
    assert (got["z"][3] == 0).all() and (got["x_out"][3] == 0).all()


def test_large_rows_do_not_overflow_early():
    t, o, dx_out, dz = make(6, 128, F, F, seed=10)
    t["x"] *= 1e12
    run_all(t, o, dx_out, dz, res_dtype=F)


def test_nan_stays_in_its_row():
    t, o, dx_out, dz = make(40, 64, F, F, seed=11)
    t["y"][7, 5] = math.nan
    x_out, z = osr.lattice_osr_norm_fwd(**t, **o)
    g = osr.lattice_osr_norm_bwd(**t, **o, dx_out=dx_out, dz=dz)
    keep = torch.arange(40, device="cuda") != 7
    for n, a in (("x_out", x_out), ("z", z), ("dy", g["dy"]), ("dgate", g["dgate"]), ("dx", g["dx"])):
        assert torch.isfinite(a[keep]).all() and torch.isnan(a[7]).all(), n


def test_in_place_residual():
    t, o, dx_out, dz = make(67, 520, BF, BF, seed=12)
    want = osr.lattice_osr_norm_fwd(**t, **o)
    gw = osr.lattice_osr_norm_bwd(**t, **o, dx_out=dx_out, dz=dz)
    d2 = dx_out.clone()
    g = osr.lattice_osr_norm_bwd(**t, **o, dx_out=d2, dz=dz,
                                 grads={**{k: torch.empty_like(v) for k, v in gw.items()}, "dx": d2})
    assert all(torch.equal(g[k], gw[k]) for k in gw)
    x = t["x"].clone()
    got = osr.lattice_osr_norm_fwd(**{**t, "x": x}, **o, x_out=x)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0].data_ptr() == x.data_ptr()


@pytest.mark.parametrize("off", [1, 4])
def test_unaligned_buffers(off):
    t, o, dx_out, dz = make(9, 264, BF, BF, seed=13)

    def shift(a):
        flat = torch.full((a.numel() + 16,), math.nan, dtype=a.dtype, device="cuda")
        v = flat[off:off + a.numel()].view(a.shape)
        v.copy_(a)
        return flat, v

    s = {k: shift(v)[1] for k, v in t.items()}
    xf, xo = shift(t["x"])
    zf, z = shift(t["y"])
    osr.lattice_osr_norm_fwd(**s, **o, x_out=xo, z=z)
    out, bound = oracle(t, o, dx_out, dz, True)
    check("x_out", xo, out["x_out"], bound["x_out"])
    check("z", z, out["z"], bound["z"])
    gw = osr.lattice_osr_norm_bwd(**t, **o, dx_out=dx_out, dz=dz, grad_dtype=BF)
    bufs = {k: shift(v) for k, v in gw.items()}
    g = osr.lattice_osr_norm_bwd(**s, **o, dx_out=shift(dx_out)[1], dz=shift(dz)[1], grad_dtype=BF,
                                 grads={k: v for k, (_, v) in bufs.items()})
    for n in g:
        check(n, g[n], out[n], bound[n])
    for flat, v in [(xf, xo), (zf, z)] + list(bufs.values()):
        assert torch.isnan(flat[:off]).all() and torch.isnan(flat[off + v.numel():]).all()


@pytest.mark.parametrize("which", ["w_post", "scale", "w_pre"])
def test_unaligned_weights(which):
    t, o, dx_out, dz = make(9, 256, BF, BF, seed=13)
    want = osr.lattice_osr_norm_bwd(**t, **o, dx_out=dx_out, dz=dz)
    t[which] = torch.cat([t[which][:1], t[which]])[1:]
    assert t[which].data_ptr() % 16 == 4
    run_all(t, o, dx_out, dz)
    assert all(torch.isfinite(v).all() for v in want.values())


def test_most_rows():
    """2^31 - 1 rows of one value: the copy a call without norms makes reaches every one of them."""
    R = 2 ** 31 - 1
    y = torch.arange(256, device="cuda").to(BF).repeat(R // 256 + 1)[:R].view(R, 1)
    x_out, z = osr.lattice_osr_norm_fwd(y, post_norm=False, pre_norm=False)
    assert z is None
    for a in range(0, R, 1 << 28):
        assert torch.equal(x_out[a:a + (1 << 28)], y[a:a + (1 << 28)])
    with pytest.raises(ValueError, match="rows"):
        osr.lattice_osr_norm_fwd(torch.empty((R + 1, 1), dtype=BF, device="cuda"), post_norm=False, pre_norm=False)


def test_empty_rows_are_refused():
    for shape in ((0, 8), (4, 0)):
        with pytest.raises(osr.OSRError) as e:
            osr.lattice_osr_norm_fwd(torch.zeros(shape, dtype=BF, device="cuda"))
        assert e.value.status == osr.ERR_SHAPE


def test_leading_dimensions():
    t, o, dx_out, dz = make(24, 40, BF, BF, seed=14)
    want = osr.lattice_osr_norm_fwd(**t, **o)
    four = {k: v.view(2, 3, 4, 40) if v.dim() == 2 else v for k, v in t.items()}
    got = osr.lattice_osr_norm_fwd(**four, **o)
    assert got[0].shape == (2, 3, 4, 40) and torch.equal(got[0].view(24, 40), want[0])


@pytest.mark.parametrize("D", [64, 2048, 5000, 10000])
def test_workspace_contents_do_not_matter(D):
    t, o, dx_out, dz = make(700, D, BF, BF, seed=18)
    want = osr.lattice_osr_norm_bwd(**t, **o, dx_out=dx_out, dz=dz)
    n = osr.lattice_osr_norm_bwd_workspace_bytes(osr.make_norm_desc(700, D, gate_kind=o["gate_kind"]))
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
    g = osr.lattice_osr_norm_bwd(**t, **o, dx_out=dx_out, dz=dz, workspace=ws[:n])
    assert all(torch.equal(g[k], want[k]) for k in want) and (ws[n:] == 255).all()


def test_reruns_streams_and_graphs():
    t, o, dx_out, dz = make(3000, 256, BF, BF, seed=15)

    def step():
        a = osr.lattice_osr_norm_fwd(**t, **o)
        g = osr.lattice_osr_norm_bwd(**t, **o, dx_out=dx_out, dz=dz)
        return [*a, *g.values()]

    first = step()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    on = osr.lattice_osr_norm_fwd(**t, **o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(on[0], first[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        new = make(3000, 256, BF, BF, seed=80 + i)[0]
        for k in t:
            t[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), i


def test_offsets_past_32_bits():
    """More than 2^31 elements in a buffer: the last rows equal a call of their own."""
    R, D = 270000, 8192
    t, o, dx_out, dz = make(64, D, BF, BF, gate=None, scale=False, seed=16)
    want = osr.lattice_osr_norm_fwd(**t, **o)
    gw = osr.lattice_osr_norm_bwd(**t, **o, dx_out=dx_out, dz=dz, grad_dtype=BF)
    big = {}
    for k in ("y", "x"):
        big[k] = torch.zeros((R, D), dtype=BF, device="cuda")
        big[k][-64:] = t[k]
    bd, bz = torch.zeros((R, D), dtype=BF, device="cuda"), torch.zeros((R, D), dtype=BF, device="cuda")
    bd[-64:], bz[-64:] = dx_out, dz
    got = osr.lattice_osr_norm_fwd(**{**t, **big}, **o)
    assert torch.equal(got[0][-64:], want[0]) and torch.equal(got[1][-64:], want[1]) and (got[1][:-64] == 0).all()
    g = osr.lattice_osr_norm_bwd(**{**t, **big}, **o, dx_out=bd, dz=bz, grad_dtype=BF)
    for k in ("dy", "dx"):
        assert torch.equal(g[k][-64:], gw[k]), k
    # rows of zeros add nothing to the column sums; only their order differs
    out, bound = oracle(t, o, dx_out, dz, True)
    for k in ("dw_post", "dw_pre"):
        check(k, g[k], out[k], bound[k])


def test_layer_forward_and_backward():
    """norm -> projections -> scan -> gated norm per head -> projection -> norm with the residual, as a block runs
    them, in fp32; every gradient against float64 differentiation of the same layer.  The bar is 1e-4 of each
    result's largest entry: fp32 products over 96 channels (96 u) through two norms and a recurrence whose gates
    average sigmoid(2), each at most some tens of units of 2^-24 times ten for the memory."""
    B, T, H, d = 2, 150, 3, 32
    D = H * d
    g = torch.Generator().manual_seed(20)
    r = lambda *s, k=1.0, m=0.0: torch.randn(s, generator=g, dtype=torch.float64) * k + m
    P = dict(x=r(B, T, D), w0=r(D, k=0.2, m=1), Wv=r(D, D, k=D ** -0.5), Wf=r(D, D, k=D ** -0.5),
             Wg=r(D, D, k=D ** -0.5), Wo=r(D, D, k=D ** -0.5), wh=r(d, k=0.2, m=1), w1=r(D, k=0.2, m=1),
             sc=r(D, k=0.1, m=0.3), w2=r(D, k=0.2, m=1), st=r(B, D))
    P = {k: v.float().double() for k, v in P.items()}
    dxo, dz, dst = r(B, T, D).float().double(), r(B, T, D).float().double(), r(B, D).float().double()

    leaf = {k: v.clone().requires_grad_() for k, v in P.items()}
    rms = lambda a: torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-6)
    z0 = leaf["x"] / rms(leaf["x"]) * leaf["w0"]
    vv, ff, gg = z0 @ leaf["Wv"], z0 @ leaf["Wf"] + 2.0, z0 @ leaf["Wg"]
    h, hs = leaf["st"], []
    for t in range(T):
        mu = torch.sigmoid(ff[:, t])
        h = mu * h + (1 - mu) * vv[:, t]
        hs.append(h)
    y = torch.stack(hs, 1).view(B, T, H, d) * torch.nn.functional.silu(gg).view(B, T, H, d)
    yh = (y / rms(y) * leaf["wh"]).reshape(B, T, D) @ leaf["Wo"]
    xo = leaf["x"] + leaf["sc"] * (yh / rms(yh) * leaf["w1"])
    z = xo / rms(xo) * leaf["w2"]
    want = torch.autograd.grad((xo * dxo).sum() + (z * dz).sum() + (h * dst).sum(), list(leaf.values()))
    want = dict(zip(leaf, want))

    p = {k: v.float().cuda() for k, v in P.items()}
    _, z0 = osr.lattice_osr_norm_fwd(None, p["x"], w_pre=p["w0"])
    vv, ff, gg = z0 @ p["Wv"], z0 @ p["Wf"] + 2.0, z0 @ p["Wg"]
    y, hT, saved = osr.lattice_osr_scan_fwd(vv, ff, p["st"], save=True)
    heads = dict(gate=gg.view(B, T, H, d), gate_kind=osr.GATE_SILU, w_post=p["wh"], pre_norm=False)
    yh, _ = osr.lattice_osr_norm_fwd(y.view(B, T, H, d), **heads)
    yo = yh.view(B, T, D) @ p["Wo"]
    block = dict(w_post=p["w1"], scale=p["sc"], w_pre=p["w2"])
    xo2, z2 = osr.lattice_osr_norm_fwd(yo, p["x"], **block)
    g1 = osr.lattice_osr_norm_bwd(yo, p["x"], dxo.float().cuda(), dz.float().cuda(), **block)
    dyh = (g1["dy"] @ p["Wo"].t()).view(B, T, H, d)
    g2 = osr.lattice_osr_norm_bwd(y.view(B, T, H, d), None, dyh, **heads)
    g3 = osr.lattice_osr_scan_bwd(vv, ff, g2["dy"].view(B, T, D), dst.float().cuda(), saved=saved)
    dgg = g2["dgate"].view(B, T, D)
    dz0 = g3["dv"] @ p["Wv"].t() + g3["dmu_logit"] @ p["Wf"].t() + dgg @ p["Wg"].t()
    g4 = osr.lattice_osr_norm_bwd(None, p["x"], g1["dx"], dz0, w_pre=p["w0"])
    flat = lambda a: a.reshape(-1, a.shape[-1])
    got = dict(x=g4["dx"], w0=g4["dw_pre"], Wv=flat(z0).t() @ flat(g3["dv"]), Wf=flat(z0).t() @ flat(g3["dmu_logit"]),
               Wg=flat(z0).t() @ flat(dgg), Wo=flat(yh.view(B, T, D)).t() @ flat(g1["dy"]), wh=g2["dw_post"],
               w1=g1["dw_post"], sc=g1["dscale"], w2=g1["dw_pre"], st=g3["dstate_in"])
    torch.cuda.synchronize()
    for n, a, b in [("x_out", xo2, xo), ("z", z2, z), ("state", hT, h)] + [(k, got[k], want[k]) for k in want]:
        err = float((a.cpu().double() - b.detach()).abs().max() / b.detach().abs().max())
        print(f"  {n}: {err:.2e}", flush=True)
        assert err <= 1e-4, (n, err)


def test_refusals_carry_the_library_s_status():
    """Forward and backward refuse alike, also where the backward's workspace is asked for first."""
    t, o, dx_out, dz = make(4, 64, BF, BF)
    wide = torch.zeros((2, 16385), dtype=BF, device="cuda")
    w = torch.ones(16385, device="cuda")
    for call in (lambda: osr.lattice_osr_norm_fwd(**t, **{**o, "eps": 0.0}),
                 lambda: osr.lattice_osr_norm_bwd(**t, **{**o, "eps": 0.0}, dx_out=dx_out, dz=dz),
                 lambda: osr.lattice_osr_norm_bwd(**t, **{**o, "gate_kind": 7}, dx_out=dx_out, dz=dz),
                 lambda: osr.lattice_osr_norm_fwd(wide, wide, w_post=w),
                 lambda: osr.lattice_osr_norm_bwd(wide, wide, wide, wide, w_post=w)):
        with pytest.raises(osr.OSRError) as e:
            call()
        assert e.value.status == osr.ERR_UNSUPPORTED


# Rows that give every workgroup of either direction (at most 768) several, none of them zeros: running column
# sums, and row sums that follow one another through the same LDS.  Vector and element layouts of every width's kernel.
MANY = [(20000, 64), (20000, 61), (9000, 200), (5000, 512), (5000, 777), (2000, 2048), (2000, 1025), (1300, 4096),
        (1300, 2050), (700, 4104), (700, 5001), (700, 8192), (700, 8200), (700, 8191), (700, 12345), (700, 16384),
        (700, 16383)]


@pytest.mark.parametrize("R,D", MANY)
@pytest.mark.parametrize("dtype", [BF, F])
def test_several_rows_per_workgroup(R, D, dtype):
    for gate in ("gelu", "silu"):
        run_all(*make(R, D, dtype, dtype, gate, seed=R + D), grad_dtype=dtype, res_dtype=dtype)


@pytest.mark.parametrize("R,D", [(9000, 96), (2000, 2000), (1300, 4000), (600, 5000), (600, 5001), (600, 9000), (600, 9001)])
@pytest.mark.parametrize("gate", ["gelu", "silu", None])
@pytest.mark.parametrize("post", [True, False])
def test_combinations_over_several_rows(R, D, gate, post):
    for x in (True, False):
        for pre in (True, False):
            for scale in (True, False):
                run_all(*make(R, D, F, F, gate, post, x, scale, pre, seed=23), res_dtype=F)


@pytest.mark.parametrize("R,D", [(2000, 2000), (600, 5000), (600, 5001), (600, 9000), (600, 9001)])
def test_types_and_absent_operands_over_several_rows(R, D):
    for in_dtype, res_dtype, grad_dtype in ((BF, F, BF), (BF, F, F), (F, BF, F), (F, BF, BF), (BF, BF, F), (F, F, BF)):
        run_all(*make(R, D, in_dtype, res_dtype, seed=24), grad_dtype=grad_dtype, res_dtype=res_dtype)
    run_all(*make(R, D, BF, BF, y=False, seed=25))
    run_all(*make(R, D, F, F, y=False, weights=False, seed=25), res_dtype=F)
    run_all(*make(R, D, BF, F, weights=False, scale=False, seed=26), res_dtype=F)
    t, o, _, dz = make(R, D, BF, BF, seed=27)
    g = osr.lattice_osr_norm_bwd(**t, **o, dx_out=None, dz=dz)
    out, bound = oracle(t, o, None, dz, True)
    for n in g:
        check(n, g[n], out[n], bound[n])


@pytest.mark.parametrize("kind", [osr.GATE_GELU, osr.GATE_SILU])
@pytest.mark.parametrize("dtype", [F, BF])
def test_gates_alone(kind, dtype):
    """phi and phi' by themselves (y, scale and the incoming gradient 1, neither norm), far into both tails."""
    g = torch.cat([torch.linspace(-13, 13, 30000), torch.linspace(-2, 2, 2768)]).view(64, 512).to(dtype).cuda()
    one = torch.ones_like(g)
    phi, _ = osr.lattice_osr_norm_fwd(one, None, gate=g, gate_kind=kind, post_norm=False, pre_norm=False, x_dtype=F)
    d = osr.lattice_osr_norm_bwd(one, None, one.float(), gate=g, gate_kind=kind, post_norm=False, pre_norm=False)
    want, dwant, rel, dabs = layer._act(kind, g)
    for name, got, ref, lim in (("phi", phi, want, rel * want.abs()), ("phi'", d["dgate"], dwant, dabs),
                                ("dy", d["dy"], want, rel * want.abs())):
        check(name, got, ref, lim + layer.TINY)


@pytest.mark.parametrize("C", [4, 16])
def test_around_the_lattice_layer(C):
    """The chunked recurrence between the norms, and the scan as the next layer: recurrence (bf16 y) -> gated norm
    of each head -> norm with the residual -> scan, and the gradients back through all of them.  Each call
    against its own oracle on what the call before it wrote: the recurrence and its gradients at their bf16 bar
    (2e-2 of the oracle's RMS), the norms and the scan element by element."""
    import numpy as np

    import oracle as osr_oracle
    from compressed_memory_linear_amd import synth
    from oracle import osr_backward

    B, T, H, m, d = 2, 64, 2, 32, 64
    D = H * d
    inp = synth.make_inputs(B, T, H, m, d, seed=1400 + C)
    t = osr.to_device(inp)
    g = torch.Generator(device="cuda").manual_seed(C)
    r = lambda *s, k=1.0, mean=0.0: torch.randn(s, generator=g, device="cuda") * k + mean
    gate, x, f = r(B, T, H, d, k=1.5).to(BF), r(B, T, D).to(BF), r(B, T, D, mean=2.0).to(BF)
    wh, w1, sc, w2 = r(d, k=0.2, mean=1), r(D, k=0.2, mean=1), r(D, k=0.1, mean=0.3), r(D, k=0.2, mean=1)
    dxo, dh, dso = r(B, T, D).to(BF), r(B, T, D).to(BF), r(B, H, m, d)

    args = [t[k] for k in ("q", "k", "v", "gamma", "mu", "state")]
    y, S = osr.lattice_osr_fwd_chunked(*args, C, y_dtype=BF)
    heads = dict(gate=gate, w_post=wh, pre_norm=False)
    yh, _ = osr.lattice_osr_norm_fwd(y, **heads)
    block = dict(w_post=w1, scale=sc, w_pre=w2)
    yb = yh.view(B, T, D)
    xo, z = osr.lattice_osr_norm_fwd(yb, x, **block)
    h, _, saved = osr.lattice_osr_scan_fwd(z, f, y_dtype=BF, save=True)
    g3 = osr.lattice_osr_scan_bwd(z, f, dh, saved=saved, grad_dtype=BF)
    g2 = osr.lattice_osr_norm_bwd(yb, x, dxo, g3["dv"], grad_dtype=BF, **block)
    g1 = osr.lattice_osr_norm_bwd(y, None, g2["dy"].view(B, T, H, d), grad_dtype=BF, **heads)
    g0 = osr.lattice_osr_bwd_chunked(*args, g1["dy"], dso, C)
    torch.cuda.synchronize()

    def rms(name, got, ref):
        err = float(np.max(np.abs(got.float().cpu().numpy() - ref)) / np.sqrt(np.mean(ref ** 2)))
        print(f"  {name}: err/rms {err:.3e}", flush=True)
        assert err <= 2e-2, (name, err)

    yr, Sr = osr_oracle.osr_forward(*inp.values_f64(), chunk_size=C)
    rms("y", y, yr)
    rms("state", S, Sr)
    ref = osr_backward.osr_backward(*inp.values_f64(), g1["dy"].float().cpu().numpy(), dso.cpu().numpy(), chunk_size=C)
    for k in ref:
        rms(k, g0[k], ref[k])

    rows = lambda a: a.reshape(-1, a.shape[-1])
    for got, out, names in (
            ({**g1, "x_out": yh}, layer.norm(rows(y), None, rows(gate), post=True, w_post=wh, pre=False,
                                             dx_out=g2["dy"].view(-1, d), backward=True),
             ("x_out", "dy", "dgate", "dw_post")),
            ({**g2, "x_out": xo, "z": z}, layer.norm(rows(yb), rows(x), None, post=True, w_post=w1, scale=sc, w_pre=w2,
                                                     dx_out=rows(dxo), dz=rows(g3["dv"]), backward=True),
             ("x_out", "z", "dy", "dx", "dw_post", "dscale", "dw_pre")),
            ({**g3, "y": h}, layer.scan(z, f, dy=dh), ("y", "dv", "dmu_logit", "dstate_in"))):
        for n in names:
            check(n, got[n], out[0][n].view(got[n].shape), out[1][n].view(got[n].shape))


def test_rows_whose_squares_pass_fp32():
    """Such a row counts as one of infinite rms: zeros behind its norm, finite, and nothing of it in other rows."""
    t, o, _, _ = make(12, 264, F, F, seed=28)
    t["x"][4] = 1e20
    x_out, z = osr.lattice_osr_norm_fwd(**t, **o)
    assert (z[4] == 0).all() and torch.isfinite(z).all() and torch.isfinite(x_out).all()
    keep = torch.arange(12, device="cuda") != 4
    out, bound = oracle(t, o)
    check("z", z[keep], out["z"][keep], bound["z"][keep])
    check("x_out", x_out, out["x_out"], bound["x_out"])


@pytest.mark.parametrize("kind", [osr.GATE_GELU, osr.GATE_SILU])
@pytest.mark.parametrize("dtype", [F, BF])
def test_gates_at_the_ends_of_the_type(kind, dtype):
    """The lowest value closes a gate and the highest opens it, with derivatives 0 and 1, and nothing becomes NaN."""
    big = torch.finfo(dtype).max
    g = torch.tensor([-big, -big / 2, -1e30, -1e4, -200.0, 200.0, 1e4, 1e30, big / 2, big] * 2, device="cuda").to(dtype)
    g = g.view(2, 10)
    one = torch.ones_like(g)
    phi, _ = osr.lattice_osr_norm_fwd(one, None, gate=g, gate_kind=kind, post_norm=False, pre_norm=False, x_dtype=F)
    d = osr.lattice_osr_norm_bwd(one, None, one.float(), gate=g, gate_kind=kind, post_norm=False, pre_norm=False)
    assert torch.equal(phi, torch.where(g > 0, g, 0).float()) and torch.equal(d["dy"], phi)
    assert torch.equal(d["dgate"], (g > 0).float())


@pytest.mark.parametrize("R,D", [(700, 64), (1300, 2048), (600, 5000), (600, 9001)])
def test_outputs_that_are_not_wanted(R, D):
    """The C calls without x_out, dx or some of the weights' gradients: the rest bit for bit, whatever is left out."""
    import ctypes

    t, o, dx_out, dz = make(R, D, BF, BF, seed=29)
    desc = osr.make_norm_desc(R, D, osr.BF16, osr.BF16, osr.F32, o["gate_kind"])
    lib, ref, ptr = osr.load_library(), ctypes.byref(desc), lambda a: None if a is None else a.data_ptr()
    st = torch.cuda.current_stream().cuda_stream
    ins = [ptr(t[k]) for k in ("y", "gate", "x", "w_post", "scale", "w_pre")]
    x_out, z = osr.lattice_osr_norm_fwd(**t, **o)
    z2 = torch.empty_like(z)
    assert lib.lattice_osr_norm_fwd(ref, *ins, None, ptr(z2), st) == osr.OK
    assert torch.equal(z, z2)
    want = osr.lattice_osr_norm_bwd(**t, **o, dx_out=dx_out, dz=dz)
    ws = torch.empty(osr.lattice_osr_norm_bwd_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    names = ("dy", "dgate", "dx", "dw_post", "dscale", "dw_pre")
    for left in (("dx",), ("dw_post",), ("dscale",), ("dw_pre",), ("dw_post", "dscale"), ("dx", "dw_post", "dscale", "dw_pre")):
        got = {k: None if k in left else torch.empty_like(want[k]) for k in names}
        sums = any(got[k] is not None for k in names[3:])
        assert lib.lattice_osr_norm_bwd(ref, *ins, ptr(dx_out), ptr(dz), *[ptr(got[k]) for k in names],
                                        ptr(ws) if sums else None, ws.numel() if sums else 0, st) == osr.OK
        assert all(got[k] is None or torch.equal(got[k], want[k]) for k in names), left
