"""The state space layer's operators together, as a layer uses them: layer norm with the residual, projection,
short convolution, projections for the steps and for B and C, scan with its gate, projection, next layer norm;
forward, backward through all of them, and token by token.

Reference: float64 on the same parameters, differentiated by torch.  Bars: every tensor between two operators
is rounded to bf16 or kept in fp32, as stated; the norm of the difference is held to the sum of those roundings'
relative sizes along the longest way, half a step of bf16 (2^-8) each; where all is fp32, to 2^-15: eighteen operators
on that way, the longest of whose sums is of 300 products, 28 roundings of 2^-24 each in the mean (a step of the
forward alone, of 10 operators and sums of 160, to 2^-17)."""
import math

import pytest
import torch

from compressed_memory_linear_amd import osr
from oracle import mixer

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
B, T, E, D, N, RANK, W = 2, 150, 96, 160, 16, 8, 4


def params(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, std=1.0: torch.randn(s, generator=g, device="cuda") * std
    return dict(w1=1 + 0.1 * r(E), b1=0.1 * r(E), win=r(E, 2 * D, std=E ** -0.5), conv=r(D, W, std=0.5), cb=0.1 * r(D),
                wx=r(D, RANK + 2 * N, std=D ** -0.5), wdt=r(RANK, D, std=RANK ** -0.5), bias=r(D) * 0.3 + math.log(math.expm1(0.05)),
                A=-torch.arange(1, N + 1, device="cuda").float() * torch.exp(0.2 * r(D, N)), skip=r(D),
                wout=r(D, E, std=D ** -0.5), w2=1 + 0.1 * r(E), b2=0.1 * r(E))


def inputs(seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, y = torch.randn((B, T, E), generator=g, device="cuda"), torch.randn((B, T, E), generator=g, device="cuda")
    seg = (torch.rand((B, T), generator=g, device="cuda") < 4 / T).cumsum(1).int()
    return x, y, seg, torch.randn((B, T, E), generator=g, device="cuda"), torch.randn((B, T, E), generator=g, device="cuda")


def layer(p, x, y, seg, dt, hist=None, state=None, lengths=None, save=False):
    """(x_out, z, tensors kept for the backward); x the residual stream (fp32), y the last layer's output (dtype dt)."""
    mm = lambda a, w: (a.float() @ w).to(dt)
    x1, z1 = osr.lattice_osr_layernorm_fwd(x, y, w=p["w1"], b=p["b1"])
    xz = mm(z1, p["win"])
    u, h1 = osr.lattice_osr_conv_fwd(xz[..., :D], p["conv"], p["cb"], hist, segments=seg, lengths=lengths, return_history=True)
    proj = mm(u, p["wx"])
    dt_ = mm(proj[..., :RANK], p["wdt"])
    Bm, Cm = proj[..., RANK:RANK + N], proj[..., RANK + N:]
    out = osr.lattice_osr_ssm_fwd(u, dt_, p["A"], Bm, Cm, state, D=p["skip"], z=xz[..., D:], dt_bias=p["bias"],
                                  segments=seg, lengths=lengths, y_dtype=dt, save=save)
    o = mm(out[0], p["wout"])
    x2, z2 = osr.lattice_osr_layernorm_fwd(x1, o, w=p["w2"], b=p["b2"])
    return x2, z2, (x1, z1, xz, u, proj, dt_, Bm, Cm, out, o, h1)


def layer_bwd(p, x, y, seg, kept, dx2, dz2, dt):
    x1, z1, xz, u, proj, dt_, Bm, Cm, out, o, _ = kept
    mm = lambda a, w: (a.float() @ w).to(dt)
    flat = lambda t: t.float().reshape(-1, t.shape[-1])
    g = {}
    n2 = osr.lattice_osr_layernorm_bwd(x1, o, dx2, dz2, w=p["w2"], b=p["b2"])
    g["w2"], g["b2"], do = n2["dw"], n2["db"], n2["dy"]
    g["wout"] = flat(out[0]).t() @ flat(do)
    s = osr.lattice_osr_ssm_bwd(u, dt_, p["A"], Bm, Cm, mm(do, p["wout"].t()), saved=out[2], D=p["skip"], z=xz[..., D:],
                                dt_bias=p["bias"], segments=seg, grad_dtype=dt)
    g["A"], g["skip"], g["bias"] = s["dA"], s["dD"], s["ddt_bias"]
    g["wdt"] = flat(proj[..., :RANK]).t() @ flat(s["ddt"])
    dproj = torch.cat([mm(s["ddt"], p["wdt"].t()), s["dB"], s["dC"]], -1)
    g["wx"] = flat(u).t() @ flat(dproj)
    du = (s["dx"].float() + dproj.float() @ p["wx"].t()).to(dt)
    c = osr.lattice_osr_conv_bwd(xz[..., :D], p["conv"], du, p["cb"], segments=seg, grad_dtype=dt)
    g["conv"], g["cb"] = c["dw"], c["dbias"]
    dxz = torch.cat([c["dx"], s["dz"]], -1)
    g["win"] = flat(z1).t() @ flat(dxz)
    n1 = osr.lattice_osr_layernorm_bwd(x, y, n2["dx"], mm(dxz, p["win"].t()), w=p["w1"], b=p["b1"])
    g["w1"], g["b1"], g["x"], g["y"] = n1["dw"], n1["db"], n1["dx"], n1["dy"]
    return g


def reference(p, x, y, seg):
    """The layer in float64 from elementary operations, the recurrence token by token."""
    ln = lambda a, w, b: (a - a.mean(-1, keepdim=True)) / torch.sqrt(a.var(-1, unbiased=False, keepdim=True) + 1e-5) * w + b
    x1 = x + y
    xz = ln(x1, p["w1"], p["b1"]) @ p["win"]
    cut = torch.zeros((B, T), dtype=torch.bool, device=x.device)
    cut[:, 1:] = seg[:, 1:] != seg[:, :-1]
    doc = cut.long().cumsum(1)
    u = p["cb"] + sum(p["conv"][:, W - 1 - k] * torch.nn.functional.pad(xz[..., :D], (0, 0, k, 0))[:, :T]
                      * (torch.nn.functional.pad(doc, (k, 0), value=0)[:, :T] == doc)[..., None] for k in range(W))
    u = u * torch.sigmoid(u)
    proj = u @ p["wx"]
    delta = torch.nn.functional.softplus(proj[..., :RANK] @ p["wdt"] + p["bias"])
    h, ys = torch.zeros((B, D, N), dtype=torch.float64, device=x.device), []
    for t in range(T):
        h = torch.where(cut[:, t, None, None], torch.zeros_like(h), h)
        h = torch.exp(delta[:, t, :, None] * p["A"]) * h + (delta * u)[:, t, :, None] * proj[:, t, None, RANK:RANK + N]
        ys.append((h * proj[:, t, None, RANK + N:]).sum(-1))
    z = xz[..., D:]
    o = ((torch.stack(ys, 1) + p["skip"] * u) * z * torch.sigmoid(z)) @ p["wout"]
    x2 = x1 + o
    return x2, ln(x2, p["w2"], p["b2"])


# Roundings to bf16 on the longest way: y, z1, xz, u, proj, dt, ssm's y, o, z2 in front; then do, its product, ddt, dproj,
# du, dx, dxz, its product and back to x.  Eighteen, each passed on at most whole in the mean.
BARS = {BF: 18 * 2.0 ** -8, F: 2.0 ** -15}


@pytest.mark.parametrize("dt", [BF, F])
def test_layer_forward_and_gradients(dt):
    p = params()
    x, y, seg, dx2, dz2 = inputs()
    y, dz2 = y.to(dt), dz2.to(dt)
    x2, z2, kept = layer(p, x, y, seg, dt, save=True)
    g = layer_bwd(p, x, y, seg, kept, dx2, dz2, dt)
    leaf = {k: t.double().requires_grad_() for k, t in dict(p, x=x, y=y).items()}
    rx, rz = reference(leaf, leaf["x"], leaf["y"], seg)
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert rel(x2, rx.detach()) <= BARS[dt] and rel(z2, rz.detach()) <= BARS[dt]
    grads = dict(zip(leaf, torch.autograd.grad((rx * dx2.double()).sum() + (rz * dz2.double()).sum(), list(leaf.values()))))
    assert set(g) == set(grads)
    for k in g:
        print(f"  {k}: {rel(g[k].reshape(grads[k].shape), grads[k]):.2e} of {BARS[dt]:.2e}", flush=True)
        assert rel(g[k].reshape(grads[k].shape), grads[k]) <= BARS[dt], k


def test_prompt_then_tokens_one_by_one():
    """A padded batch of prompts through the layer, then single tokens from the state and the history it left: what one
    call over the whole sequences gives, within the bars of fp32."""
    p = params(3)
    x, y, _, _, _ = inputs(4)
    lens = torch.tensor([97, 140], dtype=torch.int32, device="cuda")
    whole, _, _ = layer(p, x, y, None, F)
    x2, _, kept = layer(p, x, y, None, F, lengths=lens)
    hist, state = kept[10], kept[8][1]
    got = [x2[b, :n] for b, n in enumerate(lens.tolist())]
    for i in range(10):
        at = lens.long() + i
        row = lambda t: torch.stack([t[b, at[b]] for b in range(B)])[:, None]
        x1, z1 = osr.lattice_osr_layernorm_fwd(row(x), row(y), w=p["w1"], b=p["b1"])
        xz = z1 @ p["win"]
        u, _ = osr.lattice_osr_conv_step(xz[..., :D], p["conv"], hist, p["cb"], hist_out=hist)
        proj = u @ p["wx"]
        o, _ = osr.lattice_osr_ssm_step(u, proj[..., :RANK] @ p["wdt"], p["A"], proj[..., RANK:RANK + N], proj[..., RANK + N:],
                                        state, D=p["skip"], z=xz[..., D:], dt_bias=p["bias"], state_out=state)
        x3, _ = osr.lattice_osr_layernorm_fwd(x1, o @ p["wout"], w=p["w2"], b=p["b2"])
        got = [torch.cat([got[b], x3[b]]) for b in range(B)]
    for b, n in enumerate(lens.tolist()):
        err = float((got[b] - whole[b, :n + 10]).double().norm() / whole[b, :n + 10].double().norm())
        assert err <= 2.0 ** -17, (b, err)


def test_beside_the_other_recurrences():
    """The convolution and the norm around the element-wise gated recurrence: layers of both kinds share them."""
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)
    x, v, f = r(B, T, D), r(B, T, D), r(B, T, D) + 2
    w = torch.randn((D, W), generator=g, device="cuda") * 0.5
    u = osr.lattice_osr_conv_fwd(v, w)
    y, _ = osr.lattice_osr_scan_fwd(u, f.contiguous(), y_dtype=BF)
    xo, z = osr.lattice_osr_layernorm_fwd(x, y)
    from oracle import layer as other
    cu, cb = mixer.conv(v, w)
    assert float(((u.double() - cu["y"]).abs() / mixer.rounded(cb["y"], cu["y"], BF)).max()) <= 1
    so, sb = other.scan(u, f)
    assert float(((y.double() - so["y"]).abs() / mixer.rounded(sb["y"], so["y"], BF)).max()) <= 1
    lo, lb = mixer.layernorm(x.view(-1, D), y.view(-1, D))
    assert float(((z.view(-1, D).double() - lo["z"]).abs() / mixer.rounded(lb["z"], lo["z"], BF)).max()) <= 1
    assert float(((xo.view(-1, D).double() - lo["x_out"]).abs() / mixer.rounded(lb["x_out"], lo["x_out"], BF)).max()) <= 1
