"""fp64 oracle of the layer operators around the OSR recurrence: the
element-wise gated recurrence (scan) and the norms around a block, with their
gradients by hand and, for each result, a bound on what fp32 arithmetic on the
same inputs may differ by.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Torch float64, on
whatever device the inputs are; values are those of the inputs, widened exactly.

The bounds follow the arithmetic, not a run: u = 2^-24 is half a unit of fp32,
every fp32 operation is off by at most u of its result, the hardware's 2^x,
1/x, sqrt and 1/sqrt by at most 2 u.  They are first order in u and count each
rounding at the size of the sum of its operands' magnitudes, so that
cancellation is covered and no operation order is assumed.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
TINY = 1e-35  # what flushing subnormal numbers may cost

ONE, COMPLEMENT, NORM = 0, 1, 2
NONE, GELU, SILU = 0, 1, 2

# sigmoid(x) and 1 - sigmoid(x), relative: e = 2^(x log2 e) by the hardware (2 u) with the exponent's low part
# multiplied in (1 u), 1 + e (1 u), 1 / x (2 u), e s (1 u): 7 u, and 1 for what is of second order.  bf16
# logits go without the low part: |x| u more for the rounded product, and 0.23 |x| u for the rounded log2 e, which
# 2 u cover at logits of up to 8.
E_SIG = 8 * U


def _e_sig(x):
    """x as stored: its type decides how the exponent is formed."""
    if x.dtype != torch.bfloat16:
        return torch.full_like(x, E_SIG, dtype=torch.float64)
    return E_SIG + 2 * U + U * x.double().abs().clamp(max=100.0)


# ----------------------------------------------------------------- scan --
def _gates(v, f, g, weight):
    v, f = v.double(), f.double()
    mu, om = torch.sigmoid(f), torch.sigmoid(-f)
    gam = torch.sigmoid(g.double()) if g is not None else torch.ones_like(mu)
    ngam = torch.sigmoid(-g.double()) if g is not None else torch.zeros_like(mu)
    w = {ONE: torch.ones_like(mu), COMPLEMENT: om, NORM: torch.sqrt(om * (1 + mu))}[weight]
    pull = {ONE: torch.zeros_like(mu), COMPLEMENT: -mu * om, NORM: -mu * mu * torch.sqrt(om / (1 + mu))}[weight]
    return v, mu, om, gam, ngam, w, pull


def _valid(lengths, B, T, device):
    if lengths is None:
        return torch.ones((B, T, 1), dtype=torch.bool, device=device)
    n = lengths.to(device).long().clamp(0, T)
    return (torch.arange(T, device=device)[None] < n[:, None])[..., None]


def scan(v, f, g=None, state_in=None, lengths=None, weight=COMPLEMENT, dy=None, dstate_out=None):
    """h_t = mu_t h_{t-1} + w(mu_t) gamma_t v_t token by token, [B,T,D]; with dy (and dstate_out) also the
    gradient.  Returns a dict of results and a dict of bounds under the same names: y, state_out, before
    (the state before each token); dv, dmu_logit, dgamma_logit, dstate_in."""
    B, T, D = v.shape
    dev = v.device
    ok = _valid(lengths, B, T, dev)
    v, mu, om, gam, ngam, w, pull = _gates(v, f, g, weight)
    z = torch.zeros((), dtype=torch.float64, device=dev)
    es = torch.where(ok, _e_sig(f), z)                                         # of mu and 1 - mu
    eg = torch.where(ok, _e_sig(g), z) if g is not None else torch.zeros_like(es)  # of gamma
    ec = es + eg + 12 * U  # of w(mu) gamma v: both gates, a root (its own 2 u), its argument, three products
    a = torch.where(ok, mu, z + 1)
    b = torch.where(ok, w * gam * v, z)
    h = torch.zeros((B, D), dtype=torch.float64, device=dev) if state_in is None else state_in.double()
    s = h.abs()                  # the same recurrence on magnitudes
    e = torch.zeros_like(h)      # the bound on h's error
    H, before, S, E = [], [], [], []
    for t in range(T):
        before.append(h)
        S.append(s), E.append(e)
        h = a[:, t] * h + b[:, t]
        s = a[:, t] * s + b[:, t].abs()
        # a's error, the rounding of the step and of the composition of runs, b's error
        e = a[:, t] * e + torch.where(ok[:, t], (es[:, t] + ec[:, t] + 4 * U) * s, z)
        H.append(h)
    H, before, S, E = (torch.stack(x, 1) for x in (H, before, S, E))
    # the error of h after token t is that before token t + 1
    Eh = torch.cat([E[:, 1:], e[:, None]], 1)
    out = {"y": torch.where(ok, H, z), "state_out": h, "before": before}
    bound = {"y": torch.where(ok, Eh, z) + TINY, "state_out": e + TINY, "before": E + TINY}
    if dy is None:
        return out, bound
    dy = torch.where(ok, dy.double(), z)
    lam = torch.zeros((B, D), dtype=torch.float64, device=dev) if dstate_out is None else dstate_out.double()
    sl, el = lam.abs(), torch.zeros_like(lam)
    gx = gam * v
    into = mu * om * before + pull * gx
    sinto = mu * om * S + (pull * gx).abs()
    einto = mu * om * E + (4 * es + eg + 16 * U) * sinto
    names = ("dmu_logit", "dv", "dgamma_logit")
    got, lim = {n: [] for n in names}, {n: [] for n in names}
    for t in range(T - 1, -1, -1):
        lam = lam + dy[:, t]
        sl = sl + dy[:, t].abs()
        el = el + 2 * U * sl
        for n, c, ce in (("dmu_logit", into[:, t], einto[:, t]), ("dv", (w * gam)[:, t], (ec * w * gam)[:, t]),
                         ("dgamma_logit", (w * gx * ngam)[:, t], ((ec + eg) * (w * gx * ngam).abs())[:, t])):
            size = sinto[:, t] if n == "dmu_logit" else c.abs()
            got[n].append(torch.where(ok[:, t], lam * c, z))
            lim[n].append(torch.where(ok[:, t], el * size + sl * (ce + 2 * U * size), z) + TINY)
        lam, sl = a[:, t] * lam, a[:, t] * sl
        el = a[:, t] * el + torch.where(ok[:, t], (es[:, t] + 4 * U) * sl, z)
    for n in names:
        out[n] = torch.stack(got[n][::-1], 1)
        bound[n] = torch.stack(lim[n][::-1], 1)
    out["dstate_in"], bound["dstate_in"] = lam, el + TINY
    return out, bound


# ---------------------------------------------------------------- norms --
def _act(kind, g):
    """phi, phi', the relative error of phi and the absolute one of phi'.

    GeLU: Phi(-a), a = |g|, as e t q(t), e = exp(-a^2 / 2), t = 1 / (1 + 0.35 a) and a polynomial q of degree 8.
    Relative: 2.9 u for the fit (1.72e-7); t off by 3.3 u (the rounded 0.35, its product, 1 / x), which
    q(t) t passes on up to 2.28 times, and q's 8 steps and 9 rounded coefficients, together at most
    11.7 u over all a; 2 u for two products, 2 u for the hardware's 2^x: 19 u.  Its argument, two products and
    the rounded log2(e) / 2 (0.23 u): 2.23 u of a^2 / 2, so 1.125 a^2 u.  Phi(a) = 1 - Phi(-a) has one rounding more, and
    phi' = Phi + g pdf the roundings of the constant, of its product and of the sum.
    SiLU: the sigmoid's error and a product."""
    if kind == GELU:
        g = g.double()
        lower = 0.5 * torch.erfc(g.abs() * math.sqrt(0.5))
        cdf = 0.5 * torch.erfc(-g * math.sqrt(0.5))
        pdf = torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        arg = 1.125 * g * g * U
        ecdf = lower * (19 * U + arg) + torch.where(g < 0, 0.0, U) * cdf
        dphi = cdf + g * pdf
        # phi's own product is the U beside ecdf / cdf; where cdf underflows phi is below TINY
        return (g * cdf, dphi, ecdf / cdf.clamp(min=1e-300) + U,
                ecdf + (g * pdf).abs() * (4 * U + arg) + U * (dphi.abs() + ecdf))
    es = _e_sig(g)
    g = g.double()
    s, r = torch.sigmoid(g), torch.sigmoid(-g)
    return g * s, s * (1 + g * r), es + 2 * U, (3 * es + 4 * U) * s * (1 + (g * r).abs())


def norm(y=None, x=None, gate=None, gate_kind=GELU, post=True, w_post=None, scale=None, pre=True, w_pre=None, eps=1e-6,
         dx_out=None, dz=None, backward=False):
    """The norms over rows [R,D]; returns (results, bounds): x_out, z and, with backward, dy, dgate, dx,
    dw_post, dscale, dw_pre."""
    lead = y if y is not None else x
    R, D = lead.shape
    dev = lead.device
    zero = torch.zeros((), dtype=torch.float64, device=dev)
    one = zero + 1
    eps = float(torch.tensor(eps, dtype=torch.float32))
    wp = w_post.double() if w_post is not None else one
    sc = scale.double() if scale is not None else one
    wq = w_pre.double() if w_pre is not None else one
    # a sum over a row: at most 16 values a thread, 10 halvings of 1024 threads or 6 and 16 waves
    E_ROW = 48 * U
    out, bound = {}, {}
    xo = x.double() if x is not None else zero.expand(R, D)
    exo = torch.zeros((R, D), dtype=torch.float64, device=dev)
    if y is not None:
        yv = y.double()
        phi, dphi, ephi, edphi = one.expand(R, D), zero.expand(R, D), zero.expand(R, D), zero.expand(R, D)
        if gate is not None:
            phi, dphi, ephi, edphi = _act(gate_kind, gate)
        u = yv * phi
        eu = u.abs() * (ephi + 2 * U)
        r1, er1 = one.expand(R, 1), zero.expand(R, 1)  # er1: relative
        if post:
            ms = u.square().mean(-1, keepdim=True)
            r1 = (ms + eps).rsqrt()
            er1 = (u.abs() * eu).mean(-1, keepdim=True) / (ms + eps) + E_ROW / 2 + 6 * U
        n1 = u * r1
        en1 = eu * r1 + n1.abs() * (er1 + U)
        n = n1 * wp
        en = en1 * wp.abs() + n.abs() * U
        add = n * sc
        exo = en * sc.abs() + 2 * U * add.abs()
        xo = xo + add
        exo = exo + U * xo.abs()
        out["x_out"], bound["x_out"] = xo, exo + TINY
    if pre:
        ms2 = xo.square().mean(-1, keepdim=True)
        r2 = (ms2 + eps).rsqrt()
        er2 = (xo.abs() * exo).mean(-1, keepdim=True) / (ms2 + eps) + E_ROW / 2 + 6 * U
        xh = xo * r2
        exh = exo * r2 + xh.abs() * (er2 + U)
        out["z"] = xh * wq
        bound["z"] = exh * wq.abs() + 2 * U * out["z"].abs() + TINY
    if not backward:
        return out, bound

    # a column sum: rows of a thread, of a workgroup and of the second kernel
    E_COL = (R / 256 + 256) * U

    def col(a, ea):
        return a.sum(0), ea.sum(0) + E_COL * a.abs().sum(0) + TINY

    d = dx_out.double() if dx_out is not None else zero.expand(R, D)
    ed = zero.expand(R, D)
    if pre:
        dzv = dz.double()
        out["dw_pre"], bound["dw_pre"] = col(dzv * xh, dzv.abs() * (exh + 2 * U * xh.abs()))
        t = dzv * wq
        m = (t * xh).mean(-1, keepdim=True)
        em = (t.abs() * (exh + (E_ROW + 4 * U) * xh.abs())).mean(-1, keepdim=True)
        d = d + r2 * (t - xh * m)
        mag = t.abs() + (xh * m).abs()
        ed = r2 * (mag * (er2 + 6 * U) + exh * m.abs() + xh.abs() * em) + 2 * U * d.abs()
    if x is not None:
        out["dx"], bound["dx"] = d, ed + TINY
    if y is None:
        return out, bound
    out["dscale"], bound["dscale"] = col(d * n, ed * n.abs() + d.abs() * (en + 2 * U * n.abs()))
    dn, edn = d * sc, ed * sc.abs() + U * (d * sc).abs()
    out["dw_post"], bound["dw_post"] = col(dn * n1, edn * n1.abs() + dn.abs() * (en1 + 2 * U * n1.abs()))
    s, es = dn * wp, edn * wp.abs() + U * (dn * wp).abs()
    du, edu = s, es
    if post:
        m = (s * n1).mean(-1, keepdim=True)
        em = (es * n1.abs() + s.abs() * (en1 + (E_ROW + 4 * U) * n1.abs())).mean(-1, keepdim=True)
        du = r1 * (s - n1 * m)
        mag = s.abs() + (n1 * m).abs()
        edu = r1 * (es + mag * (er1 + 6 * U) + en1 * m.abs() + n1.abs() * em)
    out["dy"], bound["dy"] = du * phi, edu * phi.abs() + (du * phi).abs() * (ephi + 2 * U) + TINY
    if gate is not None:
        out["dgate"] = du * yv * dphi
        bound["dgate"] = yv.abs() * (edu * dphi.abs() + du.abs() * (edphi + 3 * U * dphi.abs())) + TINY
    return out, bound


def rounded(bound, ref, dtype):
    """The bound of an output stored in dtype: half a step of it more (fp32's own is in the bound)."""
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    return bound + half * (ref.abs() + bound)
