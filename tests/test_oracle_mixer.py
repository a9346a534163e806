"""CPU pins of the state space layer's oracle (oracle/mixer.py): its forward
against direct statements of the definitions, one scalar recurrence at a time,
its hand-written gradients against torch's differentiation of those and
against central differences."""
import pytest
import torch

from oracle import mixer

N_ = [None, [0, 5], [1, 9], [-3, 7]]


def _gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, dtype=torch.float64)


def _ssm_inputs(B=2, T=7, D=6, N=3, G=2, seed=0, gate=True, extras=True):
    r = _gen(seed)
    x = dict(x=r(B, T, D), dt=r(B, T, D), A=-r(D, N).exp(), Bm=r(B, T, G, N), Cm=r(B, T, G, N), state_in=r(B, D, N))
    if extras:
        x.update(D=r(D), dt_bias=r(D))
    if gate:
        x["z"] = r(B, T, D)
    return x, r(B, T, D), r(B, D, N)


def _ssm_loop(x, dt, A, Bm, Cm, state_in, D=None, z=None, dt_bias=None, softplus=True, lengths=None, segments=None):
    """Every channel by itself, from the definition."""
    nb, T, ch = x.shape
    G = Bm.shape[2]
    ys, states = [], []
    for b in range(nb):
        n = T if lengths is None else max(0, min(T, int(lengths[b])))
        cols, last = [], []
        for c in range(ch):
            h, col = state_in[b, c], []
            for t in range(T):
                if t >= n:
                    col.append(torch.zeros((), dtype=torch.float64))
                    continue
                if segments is not None and t and segments[b, t] != segments[b, t - 1]:
                    h = torch.zeros_like(h)
                d = dt[b, t, c] + (dt_bias[c] if dt_bias is not None else 0)
                if softplus:
                    d = torch.log(1 + torch.exp(d))
                g = c // (ch // G)
                h = torch.exp(d * A[c]) * h + d * x[b, t, c] * Bm[b, t, g]
                y = Cm[b, t, g] @ h + (D[c] * x[b, t, c] if D is not None else 0)
                col.append(y * z[b, t, c] / (1 + torch.exp(-z[b, t, c])) if z is not None else y)
            cols.append(torch.stack(col)), last.append(h)
        ys.append(torch.stack(cols, 1)), states.append(torch.stack(last))
    return torch.stack(ys), torch.stack(states)


NAMES = dict(x="dx", dt="ddt", A="dA", Bm="dB", Cm="dC", D="dD", z="dz", dt_bias="ddt_bias", state_in="dstate_in")


@pytest.mark.parametrize("gate,extras,softplus", [(True, True, True), (False, False, True), (True, True, False)])
@pytest.mark.parametrize("lengths", N_)
@pytest.mark.parametrize("packed", [False, True])
def test_ssm_matches_the_definition_and_its_gradient(gate, extras, softplus, lengths, packed):
    x, dy, dso = _ssm_inputs(gate=gate, extras=extras)
    if not softplus:
        x["dt"] = x["dt"].abs() * 0.3
        x["dt_bias"] = x["dt_bias"].abs() * 0.1
    kw = dict(softplus=softplus, lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32),
              segments=torch.tensor([[0, 0, 1, 1, 1, 4, 2], [3, 3, 3, 3, 3, 3, 3]]) if packed else None)
    out, _ = mixer.ssm(**x, **kw, dy=dy, dstate_out=dso)
    leaf = {k: t.clone().requires_grad_() for k, t in x.items()}
    y, last = _ssm_loop(**leaf, **kw)
    torch.testing.assert_close(out["y"], y.detach(), rtol=1e-11, atol=1e-12)
    torch.testing.assert_close(out["state_out"], last.detach(), rtol=1e-11, atol=1e-12)
    grads = torch.autograd.grad((y * dy).sum() + (last * dso).sum(), list(leaf.values()), allow_unused=True)
    for k, gr in zip(leaf, grads):
        torch.testing.assert_close(out[NAMES[k]], gr, rtol=1e-9, atol=1e-11)


def test_ssm_gradient_by_differences():
    x, dy, dso = _ssm_inputs(seed=3)
    kw = dict(lengths=torch.tensor([7, 5]), segments=torch.tensor([[0, 0, 0, 1, 1, 1, 1]] * 2))
    out, _ = mixer.ssm(**x, **kw, dy=dy, dstate_out=dso)

    def loss(**k):
        o, _ = mixer.ssm(**k, **kw)
        return float((o["y"] * dy).sum() + (o["state_out"] * dso).sum())

    r = _gen(9)
    for k, n in NAMES.items():
        d = r(*x[k].shape)
        num = (loss(**{**x, k: x[k] + 1e-5 * d}) - loss(**{**x, k: x[k] - 1e-5 * d})) / 2e-5
        assert num == pytest.approx(float((out[n] * d).sum()), rel=1e-6, abs=1e-7), n


def test_ssm_bounds_cover_fp32():
    """The same loop in fp32 stays inside the bounds, which are no wider than fp32 needs by orders of magnitude."""
    x, _, _ = _ssm_inputs(T=30, seed=5)
    x = {k: t.float() for k, t in x.items()}
    out, bound = mixer.ssm(**x)
    y, last = _ssm_loop(**x)
    for got, n in ((y, "y"), (last, "state_out")):
        worst = ((got.double() - out[n]).abs() / bound[n]).max()
        assert 0.005 < worst < 1, (n, worst)


def _conv_loop(x, w, bias, hist_in, act, lengths, segments):
    B, T, D = x.shape
    W = w.shape[1]
    ys, tails = [], []
    for b in range(B):
        n = T if lengths is None else max(0, min(T, int(lengths[b])))
        first = 0 if segments is None else int(segments[b, 0])
        rows = [(first, hist_in[b, i]) for i in range(W - 1)]
        start, out = 0, []  # start: the first row of the present document
        for t in range(T):
            if t >= n:
                out.append(torch.zeros(D, dtype=torch.float64))
                continue
            if segments is not None and t and segments[b, t] != segments[b, t - 1]:
                start = len(rows)
            rows.append((0, x[b, t]))
            p = bias.clone()
            for j in range(W):
                i = len(rows) - W + j
                if i >= start:
                    p = p + w[:, j] * rows[i][1]
            out.append(p / (1 + torch.exp(-p)) if act else p)
        tail = [rows[i][1] if i >= start else torch.zeros(D, dtype=torch.float64) for i in range(len(rows) - W + 1, len(rows))]
        ys.append(torch.stack(out))
        tails.append(torch.stack(tail) if tail else torch.zeros(0, D, dtype=torch.float64))
    return torch.stack(ys), torch.stack(tails)


@pytest.mark.parametrize("W", [1, 2, 4, 8])
@pytest.mark.parametrize("act", [mixer.NONE, mixer.SILU])
@pytest.mark.parametrize("lengths", N_)
@pytest.mark.parametrize("packed", [False, True])
def test_conv_matches_the_definition_and_its_gradient(W, act, lengths, packed):
    r = _gen(1)
    B, T, D = 2, 7, 3
    x = dict(x=r(B, T, D), w=r(D, W), bias=r(D), hist_in=r(B, W - 1, D))
    dy, dho = r(B, T, D), r(B, W - 1, D)
    kw = dict(act=act, lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32),
              segments=torch.tensor([[0, 0, 1, 1, 1, 4, 1], [3, 3, 3, 3, 3, 3, 3]]) if packed else None)
    out, _ = mixer.conv(**x, **kw, dy=dy, dhist_out=dho)
    leaf = {k: t.clone().requires_grad_() for k, t in x.items()}
    y, tail = _conv_loop(**leaf, **kw)
    torch.testing.assert_close(out["y"], y.detach(), rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(out["hist_out"], tail.detach(), rtol=0, atol=0)
    grads = torch.autograd.grad((y * dy).sum() + (tail * dho).sum(), list(leaf.values()), allow_unused=True)
    for k, gr in zip(leaf, grads):
        gr = torch.zeros_like(x[k]) if gr is None else gr
        torch.testing.assert_close(out["dhist_in" if k == "hist_in" else "d" + k], gr, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("affine", [False, True])
def test_layernorm_matches_the_definition_and_its_gradient(residual, affine):
    r = _gen(2)
    x = dict(x=r(5, 9) + 1)
    if residual:
        x["y"] = r(5, 9)
    if affine:
        x.update(w=r(9), b=r(9))
    dx_out, dz = r(5, 9), r(5, 9)
    out, _ = mixer.layernorm(**x, dx_out=dx_out, dz=dz)
    leaf = {k: t.clone().requires_grad_() for k, t in x.items()}
    rows = []
    for i in range(5):
        a = leaf["x"][i] + (leaf["y"][i] if residual else 0)
        mean = sum(a[j] for j in range(9)) / 9
        var = sum((a[j] - mean) ** 2 for j in range(9)) / 9
        z = (a - mean) / torch.sqrt(var + float(torch.tensor(1e-5)))
        rows.append((a, z * leaf["w"] + leaf["b"] if affine else z))
    xo, z = torch.stack([a for a, _ in rows]), torch.stack([z for _, z in rows])
    torch.testing.assert_close(out["x_out"], xo.detach(), rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(out["z"], z.detach(), rtol=1e-12, atol=1e-12)
    grads = torch.autograd.grad((xo * dx_out).sum() + (z * dz).sum(), list(leaf.values()))
    for k, gr in zip(leaf, grads):
        torch.testing.assert_close(out["dx" if k == "y" else "d" + k], gr, rtol=1e-9, atol=1e-11)
