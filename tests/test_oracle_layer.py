"""CPU pins of the layer oracle (oracle/layer.py): its forward against direct
statements of the definitions, its hand-written gradients against torch's
differentiation of them and against central differences."""
import math

import pytest
import torch

from oracle import layer

WEIGHTS = [layer.ONE, layer.COMPLEMENT, layer.NORM]


def _scan_inputs(B=2, T=7, D=5, seed=0, gamma=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    return dict(v=r(B, T, D), f=r(B, T, D) + 1, g=r(B, T, D) if gamma else None, state_in=r(B, D)), r(B, T, D), r(B, D)


def _scan_loop(v, f, g, state_in, weight, lengths=None):
    """One scalar at a time, from the definition."""
    B, T, D = v.shape
    ys, last = [], []
    for b in range(B):
        n = T if lengths is None else max(0, min(T, int(lengths[b])))
        h = state_in[b]
        rows = []
        for t in range(T):
            if t < n:
                mu = 1 / (1 + torch.exp(-f[b, t]))
                w = [torch.ones_like(mu), 1 - mu, torch.sqrt(1 - mu * mu)][weight]
                gam = 1 / (1 + torch.exp(-g[b, t])) if g is not None else 1.0
                h = mu * h + w * gam * v[b, t]
                rows.append(h)
            else:
                rows.append(torch.zeros_like(h))
        ys.append(torch.stack(rows))
        last.append(h)
    return torch.stack(ys), torch.stack(last)


@pytest.mark.parametrize("weight", WEIGHTS)
@pytest.mark.parametrize("gamma", [True, False])
@pytest.mark.parametrize("lengths", [None, [0, 4], [1, 9], [-2, 7]])
def test_scan_matches_the_definition_and_its_gradient(weight, gamma, lengths):
    x, dy, dso = _scan_inputs(gamma=gamma)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    out, _ = layer.scan(**x, lengths=n, weight=weight, dy=dy, dstate_out=dso)
    leaf = {k: t.clone().requires_grad_() for k, t in x.items() if t is not None}
    y, last = _scan_loop(leaf["v"], leaf["f"], leaf.get("g"), leaf["state_in"], weight, n)
    torch.testing.assert_close(out["y"], y.detach(), rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(out["state_out"], last.detach(), rtol=1e-12, atol=1e-12)
    grads = torch.autograd.grad((y * dy).sum() + (last * dso).sum(), list(leaf.values()), allow_unused=True)
    names = {"v": "dv", "f": "dmu_logit", "g": "dgamma_logit", "state_in": "dstate_in"}
    for k, gr in zip(leaf, grads):
        torch.testing.assert_close(out[names[k]], gr, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("weight", WEIGHTS)
def test_scan_gradient_by_differences(weight):
    x, dy, dso = _scan_inputs(seed=3)
    out, _ = layer.scan(**x, weight=weight, dy=dy, dstate_out=dso)

    def loss(**k):
        o, _ = layer.scan(**k, weight=weight)
        return float((o["y"] * dy).sum() + (o["state_out"] * dso).sum())

    g = torch.Generator().manual_seed(9)
    for k, n in (("v", "dv"), ("f", "dmu_logit"), ("g", "dgamma_logit"), ("state_in", "dstate_in")):
        d = torch.randn(x[k].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        num = (loss(**{**x, k: x[k] + h * d}) - loss(**{**x, k: x[k] - h * d})) / (2 * h)
        assert num == pytest.approx(float((out[n] * d).sum()), rel=1e-6, abs=1e-8), n


@pytest.mark.parametrize("weight", WEIGHTS)
def test_scan_saturated_gates(weight):
    """-inf drops the state, +inf keeps it and lets nothing in (but for w = 1); both have zero gradients."""
    x, dy, _ = _scan_inputs()
    x["f"][:, 3] = -math.inf
    x["f"][:, 5] = math.inf
    out, bound = layer.scan(**x, weight=weight, dy=dy)
    gv = torch.sigmoid(x["g"]) * x["v"]
    torch.testing.assert_close(out["y"][:, 3], gv[:, 3])
    torch.testing.assert_close(out["y"][:, 5], out["y"][:, 4] + (gv[:, 5] if weight == layer.ONE else 0))
    assert (out["dmu_logit"][:, [3, 5]] == 0).all() and (out["dstate_in"] != 0).any()
    assert all(torch.isfinite(t).all() for t in list(out.values()) + list(bound.values()))


CASES = [dict(), dict(gate_kind=layer.SILU), dict(gate=False), dict(post=False), dict(x=False), dict(pre=False),
         dict(x=False, pre=False), dict(weights=False), dict(y=False)]


def _norm_inputs(R=3, D=6, gate=True, x=True, y=True, post=True, pre=True, weights=True, gate_kind=layer.GELU, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    k = dict(y=r(R, D), x=r(R, D) if x else None, gate=r(R, D) if gate else None, w_post=r(D) if post else None,
             scale=r(D), w_pre=r(D) if pre else None)
    if not weights:
        k.update(w_post=None, scale=None, w_pre=None)
    if not y:
        k.update(y=None, gate=None, w_post=None, scale=None)
        post = False
    return k, dict(gate_kind=gate_kind, post=post, pre=pre, eps=1e-3), r(R, D), r(R, D) if pre else None


def _norm_definition(k, o):
    rms = lambda a: torch.sqrt((a * a).sum(-1, keepdim=True) / a.shape[-1] + float(torch.tensor(o["eps"])))
    m = k["y"]
    if m is not None:
        if k["gate"] is not None:
            act = torch.nn.functional.gelu if o["gate_kind"] == layer.GELU else torch.nn.functional.silu
            m = m * act(k["gate"])
        if o["post"]:
            m = m / rms(m)
            m = m * k["w_post"] if k["w_post"] is not None else m
        m = m * k["scale"] if k["scale"] is not None else m
    xo = k["x"] if m is None else m if k["x"] is None else k["x"] + m
    z = None
    if o["pre"]:
        z = xo / rms(xo)
        z = z * k["w_pre"] if k["w_pre"] is not None else z
    return xo, z


@pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
def test_norm_matches_the_definition_and_its_gradient(case):
    k, o, dxo, dz = _norm_inputs(**case)
    out, _ = layer.norm(**k, **o, dx_out=dxo, dz=dz, backward=True)
    leaf = {n: t.clone().requires_grad_() for n, t in k.items() if t is not None}
    xo, z = _norm_definition({**k, **leaf}, o)
    if k["y"] is not None:
        torch.testing.assert_close(out["x_out"], xo.detach(), rtol=1e-7, atol=1e-9)
    if z is not None:
        torch.testing.assert_close(out["z"], z.detach(), rtol=1e-7, atol=1e-9)
    loss = (xo * dxo).sum() + ((z * dz).sum() if z is not None else 0)
    for n, g in zip(leaf, torch.autograd.grad(loss, list(leaf.values()))):
        torch.testing.assert_close(out["d" + n], g, rtol=1e-6, atol=1e-8)


def test_norm_gradient_by_differences():
    k, o, dxo, dz = _norm_inputs(seed=4)
    out, _ = layer.norm(**k, **o, dx_out=dxo, dz=dz, backward=True)

    def loss(**kk):
        f, _ = layer.norm(**kk, **o)
        return float((f["x_out"] * dxo).sum() + (f["z"] * dz).sum())

    g = torch.Generator().manual_seed(9)
    for n in k:
        d = torch.randn(k[n].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        num = (loss(**{**k, n: k[n] + h * d}) - loss(**{**k, n: k[n] - h * d})) / (2 * h)
        assert num == pytest.approx(float((out["d" + n] * d).sum()), rel=1e-6, abs=1e-8), n


def _gate_in_fp32(x, parts):
    """sigmoid(x) and 1 - sigmoid(x) in fp32, every operation rounded: the exponent x log2(e) as one rounded product
    (parts 0), with what the product loses (1), with what the rounded log2(e) loses too (2)."""
    f32, f64 = torch.float32, torch.float64
    r = lambda a: a.to(f32).to(f64)
    x, c = -x.to(f64), r(torch.tensor(math.log2(math.e), dtype=f64))
    hi = r(x * c)
    e = r(torch.exp2(hi))
    if parts:
        lo = r(x * c - hi)
        if parts == 2:
            lo = r(x * r(math.log2(math.e) - c) + lo)
        e = r(e * r(lo * r(torch.tensor(math.log(2.0), dtype=f64))) + e)
    s = r(1 / r(1 + e))
    return s, torch.where(e > 2.0 ** 25, torch.ones_like(e), r(e * s))


def test_gate_bounds_tell_the_forms_of_the_exponent_apart():
    """The bound for fp32 logits holds the form that keeps both low parts and neither of the others; the one for
    bf16 logits holds the plain product."""
    x = torch.linspace(-80, 80, 20001)
    want = torch.sigmoid(x.double()), torch.sigmoid(-x.double())
    worst = lambda x, parts: max(float(((a / b - 1).abs() / layer._e_sig(x)).max())
                                 for a, b in zip(_gate_in_fp32(x, parts), want))
    assert worst(x, 2) < 0.6
    assert worst(x, 1) > 2 and worst(x, 0) > 6
    x = torch.linspace(-8, 8, 257).bfloat16()
    want = torch.sigmoid(x.double()), torch.sigmoid(-x.double())
    assert worst(x, 0) <= 1
