"""GPU parity of the layer norm (lattice_osr_layernorm_*) against the fp64
oracle (oracle/mixer.py), element by element, at the oracle's own bounds plus
half a step of a bf16 output."""
import math

import pytest
import torch

from compressed_memory_linear_amd import osr
from oracle import mixer

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def make(R, D, in_dtype=BF, res_dtype=BF, residual=True, affine=True, seed=0, shift=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    return dict(x=(2 * r(R, D) + shift).to(res_dtype), y=r(R, D).to(in_dtype) if residual else None,
                w=1 + 0.2 * r(D) if affine else None, b=0.2 * r(D) if affine else None), r(R, D).to(res_dtype), r(R, D).to(in_dtype)


def check(name, got, ref, bound):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), name
    worst = float((err / mixer.rounded(bound, ref, got.dtype)).max()) if err.numel() else 0.0
    print(f"  {name}: worst error / bar {worst:.3f}", flush=True)
    assert worst <= 1.0, (name, worst)


def run_all(x, dx_out, dz, grad_dtype=None, eps=1e-5):
    R, D = x["x"].shape
    print(f"layernorm R{R} D{D} x {x['x'].dtype} z {dz.dtype} residual {x['y'] is not None} affine {x['w'] is not None} "
          f"grad {grad_dtype}", flush=True)
    x_out, z = osr.lattice_osr_layernorm_fwd(x["x"], x["y"], w=x["w"], b=x["b"], eps=eps, z_dtype=dz.dtype)
    g = osr.lattice_osr_layernorm_bwd(x["x"], x["y"], dx_out, dz, w=x["w"], b=x["b"], eps=eps, grad_dtype=grad_dtype)
    out, bound = mixer.layernorm(**x, eps=eps, dx_out=dx_out, dz=dz)
    got = dict(g, z=z)
    if x["y"] is not None:
        got["x_out"] = x_out
        out["dy"], bound["dy"] = out["dx"], bound["dx"]
    else:
        assert x_out is None
    for n in got:
        check(n, got[n], out[n], bound[n])
    return got


WIDTHS = [1, 2, 7, 8, 63, 64, 65, 128, 200, 256, 511, 512, 1001, 1024, 2040, 2048, 3000, 4096, 5120, 8192, 8200, 12000, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, F])
def test_widths(D, dtype):
    run_all(*make(37, D, dtype, dtype, seed=D))


@pytest.mark.parametrize("in_dtype,res_dtype,grad_dtype", [(BF, F, None), (BF, F, BF), (F, BF, F), (BF, BF, F), (F, F, BF)])
@pytest.mark.parametrize("D", [64, 1001, 16384])
def test_types(in_dtype, res_dtype, grad_dtype, D):
    run_all(*make(19, D, in_dtype, res_dtype, seed=3), grad_dtype=grad_dtype)


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("D", [96, 1003, 9000])
def test_operands_that_may_be_left_out(residual, affine, D):
    x, dx_out, dz = make(23, D, F, F, residual, affine, seed=5)
    run_all(x, dx_out, dz)
    run_all(x, None, dz)


@pytest.mark.parametrize("R", [1, 2, 255, 256, 257, 3000, 70001])
def test_rows(R):
    run_all(*make(R, 64, seed=R))
    if R < 3000:
        run_all(*make(R, 520, BF, F, seed=R))


@pytest.mark.parametrize("shift", [100.0, 1e4])
def test_mean_far_from_zero(shift):
    """The variance comes from the differences: a mean of many deviations costs what its own rounding does."""
    run_all(*make(50, 300, F, F, residual=False, seed=7, shift=shift))
    run_all(*make(50, 2048, F, F, seed=8, shift=shift))


def test_constant_rows_and_eps():
    """Rows without variance: z = b, and gradients through 1 / sqrt(eps)."""
    x, dx_out, dz = make(20, 128, F, F, residual=False, seed=9)
    x["x"][::2] = torch.arange(10, device="cuda").float().view(-1, 1)
    for eps in (1e-5, 1.0, 1e-12):
        got = run_all(x, dx_out, dz, eps=eps)
    assert torch.equal(got["z"][0], x["b"])


def test_not_finite_values_stay_in_their_rows():
    x, dx_out, dz = make(10, 200, F, F, seed=11)
    want = osr.lattice_osr_layernorm_fwd(x["x"], x["y"], w=x["w"], b=x["b"])
    x["x"][3, 5], x["y"][6, 0] = math.nan, math.inf
    x_out, z = osr.lattice_osr_layernorm_fwd(x["x"], x["y"], w=x["w"], b=x["b"])
    g = osr.lattice_osr_layernorm_bwd(x["x"], x["y"], dx_out, dz, w=x["w"])
    keep = [i for i in range(10) if i not in (3, 6)]
    assert torch.equal(z[keep], want[1][keep]) and torch.isfinite(g["dx"][keep]).all()
    assert torch.isnan(z[[3, 6]]).all()


def test_in_place_and_shared_gradient():
    x, dx_out, dz = make(50, 256, BF, F, seed=13)
    kw = dict(w=x["w"], b=x["b"])
    want = osr.lattice_osr_layernorm_fwd(x["x"], x["y"], **kw)
    g = osr.lattice_osr_layernorm_bwd(x["x"], x["y"], dx_out, dz, **kw)
    assert g["dy"].dtype == BF and torch.equal(g["dy"], g["dx"].to(BF))
    xs = x["x"].clone()
    x_out, z = osr.lattice_osr_layernorm_fwd(xs, x["y"], x_out=xs, **kw)
    assert x_out.data_ptr() == xs.data_ptr() and torch.equal(xs, want[0]) and torch.equal(z, want[1])
    into = dict({k: torch.empty_like(t) for k, t in g.items()}, dx=dx_out.clone())
    g2 = osr.lattice_osr_layernorm_bwd(x["x"], x["y"], into["dx"], dz, grads=into, **kw)
    assert all(torch.equal(g[k], g2[k]) for k in g)
    same = make(50, 256, BF, BF, seed=14)
    g = osr.lattice_osr_layernorm_bwd(same[0]["x"], same[0]["y"], same[1], same[2], w=same[0]["w"])
    assert g["dy"] is g["dx"] and "db" not in g


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("D", [64, 2048])
def test_unaligned_buffers(off, D):
    def shifted(t):
        flat = torch.full((t.numel() + 16,), math.nan, dtype=t.dtype, device="cuda")
        view = flat[off:off + t.numel()].view(t.shape)
        view.copy_(t)
        return flat, view

    x, dx_out, dz = make(21, D, seed=15)
    s = {k: shifted(t)[1] for k, t in x.items()}
    outs = [shifted(torch.zeros_like(x["x"])) for _ in range(2)]
    osr.lattice_osr_layernorm_fwd(s["x"], s["y"], w=s["w"], b=s["b"], x_out=outs[0][1], z=outs[1][1])
    names = dict(dx=x["x"], dw=x["w"], db=x["b"])
    bufs = {k: shifted(torch.zeros_like(t)) for k, t in names.items()}
    osr.lattice_osr_layernorm_bwd(s["x"], s["y"], shifted(dx_out)[1], shifted(dz)[1], w=s["w"], b=s["b"],
                                  grads={k: v for k, (_, v) in bufs.items()})
    out, bound = mixer.layernorm(**x, dx_out=dx_out, dz=dz)
    for name, (flat, v) in dict(bufs, x_out=outs[0], z=outs[1]).items():
        check(name, v, out[name], bound[name])
        assert torch.isnan(flat[:off]).all() and torch.isnan(flat[off + v.numel():]).all(), name


def test_reruns_leading_dimensions_and_capture():
    x, dx_out, dz = make(3000, 136, BF, F, seed=17)
    kw = dict(w=x["w"], b=x["b"])

    def both(a, d, e):
        return [*osr.lattice_osr_layernorm_fwd(a["x"], a["y"], **kw),
                *osr.lattice_osr_layernorm_bwd(a["x"], a["y"], d, e, **kw).values()]

    want = both(x, dx_out, dz)
    assert all(torch.equal(a, b) for a, b in zip(want, both(x, dx_out, dz)))
    four = {k: t.view(10, 300, 136) for k, t in x.items() if k in "xy"}
    got = both(four, dx_out.view(10, 300, 136), dz.view(10, 300, 136))
    assert all(torch.equal(a, b.reshape(a.shape)) for a, b in zip(want, got))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(x, dx_out, dz)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(x, dx_out, dz)
    for _ in range(3):
        for t in got:
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        both(x, dx_out, dz)
        torch.cuda.synchronize()
