"""fp64 oracle of the selective state space layer: its scan, the short causal
convolution in front of it and the layer norm around it, with their gradients
by hand and, for each result, a bound on what fp32 arithmetic on the same
inputs may differ by.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Torch float64, on
whatever device the inputs are; values are those of the inputs, widened exactly.
The bounds are made as in oracle/layer.py: first order in u = 2^-24, every
rounding at the size of the sum of its operands' magnitudes, hardware 2^x and
1/x at 2 u, sums at the depth of their longest chain of additions.
"""
from __future__ import annotations

import torch

from .layer import E_SIG, TINY, U, rounded  # noqa: F401  (rounded: for the tests)

NONE, SILU = 0, 1

# softplus beside the rounding of its argument: e = exp(-|v|) 4 u (as in E_SIG); t = e / (2 + e): 4 u more, which
# atanh passes on up to 1.13 times; the polynomial's last steps, its coefficients and its fit 2.5 u; the product
# and the sum 2 u.
E_SOFTPLUS = 16 * U


def _exponent(v, bf16):
    """What the exponential of v is off by beside the hardware's error: for bf16 inputs its exponent is one rounded
    product with a rounded log2(e), 1.25 |v| u (as in oracle/layer.py); for fp32 ones it keeps what these lose."""
    return 2 * U + 1.25 * U * v.abs().clamp(max=100.0) if bf16 else torch.zeros_like(v)


def _silu(z, bf16=False):
    """phi, phi' and their absolute errors."""
    s, r = torch.sigmoid(z), torch.sigmoid(-z)
    es = E_SIG + _exponent(z, bf16)
    return z * s, s * (1 + z * r), (es + 2 * U) * (z * s).abs(), (3 * es + 4 * U) * s * (1 + (z * r).abs())


def _tokens(lengths, segments, B, T, device):
    """[B,T] truth values: tokens, and tokens that begin a document."""
    ok = torch.ones((B, T), dtype=torch.bool, device=device)
    if lengths is not None:
        ok = torch.arange(T, device=device)[None] < lengths.to(device).long().clamp(0, T)[:, None]
    cut = torch.zeros((B, T), dtype=torch.bool, device=device)
    if segments is not None:
        cut[:, 1:] = segments[:, 1:] != segments[:, :-1]
    return ok, cut & ok


# ------------------------------------------------------------------ ssm --
def ssm(x, dt, A, Bm, Cm, state_in=None, D=None, z=None, dt_bias=None, softplus=True, lengths=None, segments=None,
        dy=None, dstate_out=None):
    """The scan token by token; with dy (and dstate_out) also the gradient.  x, dt, z [B,T,D], Bm, Cm [B,T,G,N].
    Returns a dict of results and one of bounds: y, state_out; dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dstate_in."""
    nb, T, ch = x.shape
    G, N = Bm.shape[2:]
    dev, K = x.device, ch // G
    f8 = torch.float64
    zero = torch.zeros((), dtype=f8, device=dev)
    ok, cut = _tokens(lengths, segments, nb, T, dev)
    on = lambda t: torch.where(ok.view(nb, T, *([1] * (t.dim() - 2))), t, zero)
    bf16 = dt.dtype == torch.bfloat16
    x, A = on(x.double()), A.double()
    raw = on(dt.double())
    eraw = torch.zeros_like(raw)
    if dt_bias is not None:
        raw = on(raw + dt_bias.double())
        eraw = U * raw.abs()
    if softplus:
        slope = torch.sigmoid(raw)
        delta = on(raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs())))
        ee = _exponent(raw, bf16)
        edelta = (E_SOFTPLUS + ee) * delta + slope * eraw
        eslope = slope * (E_SIG + ee + torch.sigmoid(-raw) * eraw)
    else:
        slope, delta, edelta, eslope = torch.ones_like(raw), raw, eraw, torch.zeros_like(raw)
    u = delta * x
    eu = edelta * x.abs() + U * u.abs()
    wide = lambda m, t: on(m.double())[:, t].repeat_interleave(K, dim=1)  # [B,D,N]
    dsk = D.double() if D is not None else torch.zeros(ch, dtype=f8, device=dev)
    phi = dphi = torch.ones_like(x)
    ephi = edphi = torch.zeros_like(x)
    if z is not None:
        phi, dphi, ephi, edphi = _silu(on(z.double()), bf16)

    def decay(t):
        """exp(delta A) and its error: A log2 e and the product 2.3 u of the exponent, the steps' own error, those of
        a run's sum of steps (taken in parts of 8, then in fp64) 9 u, 2^x 2 u."""
        e = delta[:, t, :, None] * A
        a = torch.exp(e)
        ea = a * (14 * U * e.abs() + A.abs() * edelta[:, t, :, None] + 2 * U)
        keep = (~cut[:, t])[:, None, None]
        return torch.where(keep, a, zero), torch.where(keep, ea, zero)

    h = torch.zeros((nb, ch, N), dtype=f8, device=dev) if state_in is None else state_in.double()
    s, e = h.abs(), torch.zeros_like(h)  # the recurrence on magnitudes, the bound on h's error
    H, S, E, core, ecore = [], [], [], [], []
    for t in range(T):
        H.append(h), S.append(s), E.append(e)
        a, ea = decay(t)
        Bt, Ct = wide(Bm, t), wide(Cm, t)
        b = u[:, t, :, None] * Bt
        live = ok[:, t, None, None]
        e2 = a * e + ea * s + eu[:, t, :, None] * Bt.abs() + U * b.abs()
        h, s2 = a * h + b, a * s + b.abs()
        e = torch.where(live, e2 + 3 * U * s2, e)
        s = s2
        core.append((h * Ct).sum(-1))
        ecore.append((Ct.abs() * (e + (N + 4) * U * s)).sum(-1))
    core, ecore = torch.stack(core, 1), torch.stack(ecore, 1)
    add = dsk * x
    ecore = ecore + 2 * U * (core.abs() + add.abs())
    core = core + add
    out = {"y": on(core * phi), "state_out": h}
    bound = {"y": on(ecore * phi.abs() + core.abs() * ephi + 2 * U * (core * phi).abs()) + TINY, "state_out": e + TINY}
    if dy is None:
        return out, bound
    H.append(h), S.append(s), E.append(e)
    dy = on(dy.double())
    if z is not None:
        out["dz"] = on(dy * core * dphi)
        bound["dz"] = on(dy.abs() * (ecore * dphi.abs() + core.abs() * (edphi + 3 * U * dphi.abs()))) + TINY
    g = dy * phi
    eg = dy.abs() * ephi + U * g.abs() if z is not None else torch.zeros_like(g)
    lam = torch.zeros_like(h) if dstate_out is None else dstate_out.double()
    sl, el = lam.abs(), torch.zeros_like(lam)
    narrow = lambda t: t.view(nb, G, K, N).sum(2)
    E_CH = (12 + (K + 63) // 64) * U  # sums over a group's channels: a product, 64 lanes, the blocks in turn
    E_TOK = (T + 64 + nb) * U         # sums over tokens: one lane's in turn, waves, sequences
    rows = {k: [] for k in ("dB", "eB", "dC", "eC", "du", "edu", "q", "eq")}
    dA, eA = torch.zeros_like(A), torch.zeros_like(A)
    for t in range(T - 1, -1, -1):
        live = ok[:, t, None, None]
        a, ea = decay(t)
        Bt, Ct = wide(Bm, t), wide(Cm, t)
        gt, egt, ut, eut = g[:, t, :, None], eg[:, t, :, None], u[:, t, :, None], eu[:, t, :, None]
        lam, sl = lam + Ct * gt, sl + (Ct * gt).abs()
        el = torch.where(live, el + Ct.abs() * egt + 2 * U * sl, el)
        h1, s1, e1 = H[t + 1], S[t + 1], E[t + 1]
        rows["dC"].append(narrow(gt * h1))
        rows["eC"].append(narrow(gt.abs() * (e1 + E_CH * s1) + egt * s1))
        rows["dB"].append(narrow(lam * ut))
        rows["eB"].append(narrow(ut.abs() * (el + E_CH * sl) + sl * eut))
        rows["du"].append((lam * Bt).sum(-1))
        rows["edu"].append((Bt.abs() * (el + (N + 4) * U * sl)).sum(-1))
        r, sr = a * lam, a * sl
        er = torch.where(live, a * el + ea * sl + 3 * U * sr, el)
        k = r * H[t]
        mag = sr * S[t]
        ek = er * S[t] + sr * E[t] + U * mag
        rows["q"].append((k * A).sum(-1))
        rows["eq"].append((A.abs() * (ek + (N + 8) * U * mag)).sum(-1))
        d4, ed4 = delta[:, t, :, None], edelta[:, t, :, None]
        dA = dA + (k * d4).sum(0)
        eA = eA + (d4 * (ek + E_TOK * mag) + ed4 * mag).sum(0)
        lam, sl, el = r, sr, er
    rows = {k: torch.stack(v[::-1], 1) for k, v in rows.items()}
    out["dB"], bound["dB"] = on(rows["dB"]), on(rows["eB"]) + TINY
    out["dC"], bound["dC"] = on(rows["dC"]), on(rows["eC"]) + TINY
    out["dA"], bound["dA"] = dA, eA + TINY
    out["dstate_in"], bound["dstate_in"] = lam, el + TINY
    du, edu = rows["du"], rows["edu"]
    out["dx"] = on(du * delta + dsk * g)
    bound["dx"] = on(edu * delta + du.abs() * edelta + dsk.abs() * eg + 2 * U * ((du * delta).abs() + (dsk * g).abs())) + TINY
    dd = rows["q"] + du * x
    edd = rows["eq"] + edu * x.abs() + 2 * U * (rows["q"].abs() + (du * x).abs())
    out["ddt"] = on(dd * slope)
    bound["ddt"] = on(edd * slope + dd.abs() * (eslope + U * slope)) + TINY
    if dt_bias is not None:
        out["ddt_bias"] = out["ddt"].sum((0, 1))
        bound["ddt_bias"] = (bound["ddt"] + E_TOK * out["ddt"].abs()).sum((0, 1))
    if D is not None:
        out["dD"] = (g * x).sum((0, 1))
        bound["dD"] = (eg * x.abs() + E_TOK * (g * x).abs()).sum((0, 1)) + TINY
    return out, bound


# ----------------------------------------------------------------- conv --
def conv(x, w, bias=None, hist_in=None, act=SILU, lengths=None, segments=None, dy=None, dhist_out=None):
    """The convolution by taps; with dy (and dhist_out) also the gradient.  Returns results and bounds: y, hist_out; dx,
    dw, dbias, dhist_in."""
    B, T, D = x.shape
    W = w.shape[1]
    dev = x.device
    zero = torch.zeros((), dtype=torch.float64, device=dev)
    ok, cut = _tokens(lengths, segments, B, T, dev)
    on = lambda t: torch.where(ok[..., None], t, zero)
    w = w.double()
    hist = torch.zeros((B, W - 1, D), dtype=torch.float64, device=dev) if hist_in is None else hist_in.double()
    rows = torch.cat([hist, on(x.double())], 1)  # row t + W - 1 is token t
    # the number of borders up to each row: a tap counts where its row's is the token's own
    doc = torch.cat([torch.zeros((B, W - 1), dtype=torch.long, device=dev), cut.long().cumsum(1)], 1)
    same = [(doc[:, j:j + T] == doc[:, W - 1:])[..., None] for j in range(W)]
    tap = [torch.where(same[j], rows[:, j:j + T], zero) for j in range(W)]
    p = sum(tap[j] * w[:, j] for j in range(W))
    mag = sum((tap[j] * w[:, j]).abs() for j in range(W))
    if bias is not None:
        p, mag = p + bias.double(), mag + bias.double().abs()
    ep = (W + 1) * U * mag
    phi, dphi, ephi, edphi = _silu(p, x.dtype == torch.bfloat16) if act == SILU else (p, torch.ones_like(p), torch.zeros_like(p), torch.zeros_like(p))
    n = torch.full((B,), T, device=dev) if lengths is None else lengths.to(dev).long().clamp(0, T)
    at = n[:, None] + torch.arange(W - 1, device=dev)  # the rows behind the last token
    alive = (torch.gather(doc, 1, at) == torch.gather(doc, 1, (n + W - 2)[:, None])) if W > 1 else at.bool()
    idx = at[..., None].expand(-1, -1, D)
    tail = torch.where(alive[..., None], torch.gather(rows, 1, idx), zero)
    # |phi'| <= 1.1 and |phi''| <= 0.5
    out = {"y": on(phi), "hist_out": tail}
    bound = {"y": on(1.1 * ep + ephi) + TINY, "hist_out": torch.zeros_like(tail) + TINY}
    if dy is None:
        return out, bound
    dy = on(dy.double())
    dp = dy * dphi
    edp = dy.abs() * (edphi + 0.5 * ep + (U * dphi.abs() if act == SILU else 0))
    drows, erows, mrows = (torch.zeros_like(rows) for _ in range(3))
    for j in range(W):
        drows[:, j:j + T] += torch.where(same[j], dp * w[:, j], zero)
        mrows[:, j:j + T] += torch.where(same[j], (dp * w[:, j]).abs(), zero)
        erows[:, j:j + T] += torch.where(same[j], edp * w[:, j].abs(), zero)
    if dhist_out is not None and W > 1:
        back = torch.where(alive[..., None], dhist_out.double(), zero)
        drows.scatter_add_(1, idx, back)
        mrows.scatter_add_(1, idx, back.abs())
    erows += (W + 2) * U * mrows
    out["dx"], bound["dx"] = on(drows[:, W - 1:]), on(erows[:, W - 1:]) + TINY
    out["dhist_in"], bound["dhist_in"] = drows[:, :W - 1], erows[:, :W - 1] + TINY
    E_TOK = (256 + B * T / 32) * U  # a run's tokens in turn, then the runs' sums
    out["dw"] = torch.stack([(dp * tap[j]).sum((0, 1)) for j in range(W)], -1)
    bound["dw"] = torch.stack([((edp + E_TOK * dp.abs()) * tap[j].abs()).sum((0, 1)) for j in range(W)], -1) + TINY
    # a sum whose terms together pass fp32's range may do so in any order of adding
    total = torch.stack([(dp * tap[j]).abs().sum((0, 1)) for j in range(W)], -1)
    bound["dw"] = torch.where(total < torch.finfo(torch.float32).max, bound["dw"], torch.inf)
    out["dbias"], bound["dbias"] = dp.sum((0, 1)), (edp + E_TOK * dp.abs()).sum((0, 1)) + TINY
    return out, bound


# ----------------------------------------------------------- layer norm --
def layernorm(x, y=None, w=None, b=None, eps=1e-5, dx_out=None, dz=None):
    """The layer norm over rows [R,D]; with dz (and dx_out) also the gradient.  Returns results and bounds:
    x_out, z; dx, dw, db."""
    R, D = x.shape
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    E_ROW = 48 * U  # a sum over a row, as for the other norms
    x = x.double()
    ex = zero
    if y is not None:
        x = x + y.double()
        ex = U * x.abs()
    m = x.mean(-1, keepdim=True)
    em = (ex + (E_ROW + 2 * U) * x.abs()).mean(-1, keepdim=True)
    c = x - m
    ec = ex + em + U * c.abs()
    var = c.square().mean(-1, keepdim=True)
    r = (var + eps).rsqrt()
    er = (c.abs() * ec).mean(-1, keepdim=True) / (var + eps) + E_ROW / 2 + 6 * U  # relative
    n = c * r
    en = ec * r + n.abs() * (er + U)
    wv = w.double() if w is not None else zero + 1
    bv = b.double() if b is not None else zero
    out = {"x_out": x, "z": n * wv + bv}
    bound = {"x_out": ex + zero.expand(R, D) + TINY, "z": en * wv.abs() + U * out["z"].abs() + TINY}
    if dz is None:
        return out, bound
    E_COL = (R / 256 + 256) * U
    dz = dz.double()
    out["dw"], bound["dw"] = (dz * n).sum(0), (dz.abs() * (en + (E_COL + 2 * U) * n.abs())).sum(0) + TINY
    out["db"], bound["db"] = dz.sum(0), E_COL * dz.abs().sum(0) + TINY
    t = dz * wv
    mt, emt = t.mean(-1, keepdim=True), ((E_ROW + 4 * U) * t.abs()).mean(-1, keepdim=True)
    mn = (t * n).mean(-1, keepdim=True)
    emn = (t.abs() * (en + (E_ROW + 6 * U) * n.abs())).mean(-1, keepdim=True)
    mag = t.abs() + mt.abs() + (n * mn).abs()
    d = r * (t - mt - n * mn)
    ed = r * (U * t.abs() + emt + en * mn.abs() + n.abs() * emn + mag * (er + 6 * U))
    if dx_out is not None:
        d = d + dx_out.double()
    out["dx"], bound["dx"] = d, ed + 2 * U * d.abs() + TINY
    return out, bound
