"""What is timed of the element-wise gated recurrence (scan) and of the norms
around a block: the cases, their inputs, one pass through each and its exact
result.

    scan   mu = sigmoid(mu_logit), gamma = sigmoid(gamma_logit) (or 1),
           h_t = mu_t h_{t-1} + w(mu_t) gamma_t v_t,  y_t = h_t,
           w(mu) = 1 ("one"), 1 - mu ("complement") or sqrt(1 - mu^2) ("norm")
    norms  u = y phi(gate),  n = u / rms(u) w_post,  x' = x + scale n,
           z = x' / rms(x') w_pre,  rms(a) = sqrt(mean(a^2) + eps) over a row

``own`` chooses between the plain form (elementary torch operations in 32 bits)
and the calls of this package.
"""
import math

import torch

own = False

EPS = 1e-6
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases --
def listed():
    return [
        # one layer's prefill over eight sequences of 4096 tokens, 16 heads of 128 channels: the ordinary call
        {"name": "scan_prefill_b8_t4096_d2048", "op": "scan_prefill", "B": 8, "T": 4096, "D": 2048, "dtype": "bf16",
         "y_dtype": "bf16", "weight": "complement", "gamma": False, "ragged": False, "resets": False, "mean": 2.0},
        # one long document, 16 heads of 128: few rows, the time axis has to fill the chip; with the writing intensity
        {"name": "scan_prefill_b1_t65536_d2048", "op": "scan_prefill", "B": 1, "T": 65536, "D": 2048, "dtype": "bf16",
         "y_dtype": "bf16", "weight": "norm", "gamma": True, "ragged": False, "resets": False, "mean": 3.0},
        # a padded batch of prompts of different lengths (one empty, one of a single token), odd sizes, fp32
        {"name": "scan_prefill_padded_b7_t1531_d1001", "op": "scan_prefill", "B": 7, "T": 1531, "D": 1001,
         "dtype": "f32", "y_dtype": "f32", "weight": "one", "gamma": True, "ragged": True, "resets": False,
         "mean": 2.0},
        # a training step of the same layer as the first case, documents packed behind one another (the state is
        # dropped at their borders by a forget logit of minus infinity): forward and all gradients
        {"name": "scan_train_b8_t4096_d2048", "op": "scan_train", "B": 8, "T": 4096, "D": 2048, "dtype": "bf16",
         "y_dtype": "bf16", "weight": "complement", "gamma": True, "ragged": False, "resets": True, "mean": 2.0},
        # training on one long document: the largest call
        {"name": "scan_train_b1_t65536_d2048", "op": "scan_train", "B": 1, "T": 65536, "D": 2048, "dtype": "bf16",
         "y_dtype": "bf16", "weight": "complement", "gamma": False, "ragged": False, "resets": False, "mean": 3.0},
        # a small fp32 training step at odd sizes, as when a model is tried out
        {"name": "scan_train_b3_t777_d513", "op": "scan_train", "B": 3, "T": 777, "D": 513, "dtype": "f32",
         "y_dtype": "f32", "weight": "norm", "gamma": True, "ragged": False, "resets": False, "mean": 2.0},
        # one new token for each of 256 sequences, 32 heads of 128: the serving step of a full batch
        {"name": "scan_step_b256_d4096", "op": "scan_step", "B": 256, "T": 1, "D": 4096, "dtype": "bf16",
         "y_dtype": "bf16", "weight": "complement", "gamma": True, "ragged": False, "resets": False, "mean": 2.0},
        # one new token for one sequence: the smallest call, where only latency counts
        {"name": "scan_step_b1_d2048", "op": "scan_step", "B": 1, "T": 1, "D": 2048, "dtype": "bf16",
         "y_dtype": "bf16", "weight": "complement", "gamma": True, "ragged": False, "resets": False, "mean": 2.0},
        # between two blocks in training or prefill: gate, norm of the block's output, residual, norm before the next
        {"name": "norm_fwd_r32768_d2048", "op": "norm_fwd", "R": 32768, "D": 2048, "dtype": "bf16",
         "res_dtype": "bf16", "gate": "gelu", "post": True, "residual": True, "scale": True, "pre": True},
        # the same for the 256 tokens of one decoding step of a wider model, residual stream in fp32
        {"name": "norm_fwd_r256_d4096", "op": "norm_fwd", "R": 256, "D": 4096, "dtype": "bf16",
         "res_dtype": "f32", "gate": "gelu", "post": True, "residual": True, "scale": True, "pre": True},
        # the backward of the first norm case
        {"name": "norm_bwd_r32768_d2048", "op": "norm_bwd", "R": 32768, "D": 2048, "dtype": "bf16",
         "res_dtype": "bf16", "gate": "gelu", "post": True, "residual": True, "scale": True, "pre": True},
        # the backward of a gated norm over each head of 64 channels (4 x 2048 tokens, 8 heads): many short rows
        {"name": "norm_bwd_heads_r65536_d64", "op": "norm_bwd", "R": 65536, "D": 64, "dtype": "bf16",
         "res_dtype": "bf16", "gate": "silu", "post": True, "residual": False, "scale": False, "pre": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if rng.random() < 0.6:
        op = rng.choice(["scan_prefill", "scan_train", "scan_step"])
        B = _log_int(rng, 1, 512 if op == "scan_step" else 32)
        T = 1 if op == "scan_step" else _log_int(rng, 1, 65536)
        D = _log_int(rng, 16, 8192)
        if rng.random() < 0.6:
            D = max(16, D // 16 * 16)
        most = 24_000_000  # elements of one tensor: well under the largest listed case
        while B * T * D > most:
            if B > 1 and rng.random() < 0.5:
                B = (B + 1) // 2
            elif T > 1:
                T = (T + 1) // 2
            else:
                D = (D + 1) // 2
        return {"op": op, "B": B, "T": T, "D": D, "dtype": dtype, "y_dtype": rng.choice([dtype, "f32"]),
                "weight": rng.choice(["one", "complement", "norm"]), "gamma": rng.random() < 0.5,
                "ragged": op != "scan_step" and rng.random() < 0.4, "resets": op != "scan_step" and rng.random() < 0.3,
                "mean": rng.choice([1.0, 2.0, 3.0])}
    D = _log_int(rng, 16, 8192)
    if rng.random() < 0.7:
        D = max(16, D // 16 * 16)
    R = _log_int(rng, 1, max(1, min(100_000, 24_000_000 // D)))
    post, residual, pre = rng.random() < 0.8, rng.random() < 0.8, rng.random() < 0.8
    post = post or not (residual or pre)
    return {"op": rng.choice(["norm_fwd", "norm_bwd"]), "R": R, "D": D, "dtype": dtype,
            "res_dtype": rng.choice([dtype, "f32"]), "gate": rng.choice(["none", "gelu", "silu"]), "post": post,
            "residual": residual, "scale": residual and rng.random() < 0.5, "pre": pre}


# --------------------------------------------------------------- inputs --
def prepare(case, seed):
    """Activations of unit size, forget logits N(mean, 1) as the gates of a trained recurrence sit, norm weights
    around 1 and residual scales around 0.3; everything from the seed alone."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape, mean=0.0, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dtype)

    s = {"case": dict(case)}
    if case["op"].startswith("scan"):
        B, T, D = case["B"], case["T"], case["D"]
        yt = _DT[case["y_dtype"]]
        s["v"] = normal(B, T, D)
        s["mu_logit"] = normal(B, T, D, mean=case["mean"])
        if case["resets"]:  # document borders, a few in every sequence
            border = torch.rand((B, T, 1), generator=g, device=dev) < 4.0 / max(T, 4)
            s["mu_logit"].masked_fill_(border, float("-inf"))
        s["gamma_logit"] = normal(B, T, D) if case["gamma"] else None
        s["state_in"] = normal(B, D, dtype=torch.float32)
        s["lengths"] = None
        if case["ragged"]:
            n = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
            if B >= 3:
                n[0], n[1], n[2] = 0, 1, T
            s["lengths"] = n
        if case["op"] == "scan_train":
            s["dy"] = normal(B, T, D, dtype=yt)
            s["dstate_out"] = normal(B, D, dtype=torch.float32)
        if case["op"] == "scan_step":  # a serving loop keeps its output buffers
            s["y"] = torch.empty((B, T, D), dtype=yt, device=dev)
            s["state_out"] = torch.empty((B, D), device=dev)
        return s
    R, D = case["R"], case["D"]
    rt = _DT[case["res_dtype"]]
    s["y"] = normal(R, D)
    s["gate"] = normal(R, D, std=1.5) if case["gate"] != "none" else None
    s["x"] = normal(R, D, std=2.0, dtype=rt) if case["residual"] else None
    s["w_post"] = normal(D, mean=1.0, std=0.2, dtype=torch.float32) if case["post"] else None
    s["scale"] = normal(D, mean=0.3, std=0.1, dtype=torch.float32) if case["scale"] else None
    s["w_pre"] = normal(D, mean=1.0, std=0.2, dtype=torch.float32) if case["pre"] else None
    if case["op"] == "norm_bwd":
        s["dx_out"] = normal(R, D, dtype=rt)
        s["dz"] = normal(R, D) if case["pre"] else None
    return s


# ------------------------------------------------------- the plain form --
def _plain_linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0, by doubling."""
    a, b = a.clone(), b.clone()
    s = 1
    while s < a.shape[1]:
        b[:, s:] += a[:, s:] * b[:, :-s]
        a[:, s:] = a[:, s:] * a[:, :-s]
        s *= 2
    return b


def _plain_gates(s):
    c = s["case"]
    f = s["mu_logit"].float()
    mu, om = 1 / (1 + torch.exp(-f)), 1 / (1 + torch.exp(f))
    gamma = 1 / (1 + torch.exp(-s["gamma_logit"].float())) if c["gamma"] else None
    w = {"one": lambda: torch.ones_like(mu), "complement": lambda: om,
         "norm": lambda: torch.sqrt(om * (1 + mu))}[c["weight"]]()
    x = s["v"].float()
    return mu, om, w, gamma, x, (x * gamma if gamma is not None else x)


def _plain_valid(s):
    T = s["v"].shape[1]
    if s["lengths"] is None:
        return None
    return (torch.arange(T, device=s["v"].device)[None] < s["lengths"][:, None])[..., None]


def _plain_scan(s):
    """The hidden states in 32 bits, with what they came from."""
    mu, om, w, gamma, x, gx = _plain_gates(s)
    ok = _plain_valid(s)
    b = w * gx
    a = mu
    if ok is not None:  # a padded token keeps the state
        a, b = torch.where(ok, mu, 1.0), torch.where(ok, b, 0.0)
    first = b.clone()
    first[:, 0] += a[:, 0] * s["state_in"]
    return _plain_linear_scan(a, first), (a, ok, mu, om, w, gamma, x, gx)


def _plain_scan_forward(s):
    h, more = _plain_scan(s)
    ok = more[1]
    y = h if ok is None else torch.where(ok, h, 0.0)
    return y.to(_DT[s["case"]["y_dtype"]]), h[:, -1].clone(), h, more


def _plain_scan_train(s):
    c = s["case"]
    y, last, h, (a, ok, mu, om, w, gamma, x, gx) = _plain_scan_forward(s)
    dy = s["dy"].float()
    if ok is not None:
        dy = torch.where(ok, dy, 0.0)
    dy = dy.clone()
    dy[:, -1] += s["dstate_out"]
    nxt = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    lam = _plain_linear_scan(nxt.flip(1), dy.flip(1)).flip(1)
    before = torch.cat([s["state_in"][:, None], h[:, :-1]], 1)
    into = mu * om * before
    if c["weight"] == "complement":
        into = into - mu * om * gx
    elif c["weight"] == "norm":
        into = into - mu * mu * torch.sqrt(om / (1 + mu)) * gx
    g = {"y": y, "state_out": last, "dmu_logit": lam * into}
    g["dv"] = lam * w * gamma if gamma is not None else lam * w
    if gamma is not None:
        g["dgamma_logit"] = lam * w * gx * (1 - gamma)
    for n in ("dmu_logit", "dv", "dgamma_logit"):
        if n in g:
            if ok is not None:
                g[n] = torch.where(ok, g[n], 0.0)
            g[n] = g[n].to(_DT[c["dtype"]])
    g["dstate_in"] = a[:, 0] * lam[:, 0]
    return g


def _plain_act(kind, g):
    """phi(g) and its derivative."""
    if kind == "gelu":
        cdf = 0.5 * torch.erfc(-g * math.sqrt(0.5))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    sg = 1 / (1 + torch.exp(-g))
    return g * sg, sg * (1 + g * (1 - sg))


def _plain_norm_parts(s):
    c = s["case"]
    y = s["y"].float()
    phi, dphi = _plain_act(c["gate"], s["gate"].float()) if c["gate"] != "none" else (None, None)
    u = y * phi if phi is not None else y
    r1 = n1 = None
    n = u
    if c["post"]:
        r1 = 1 / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS)
        n1 = u * r1
        n = n1 * s["w_post"]
    xo = n * s["scale"] if c["scale"] else n
    if c["residual"]:
        xo = xo + s["x"].float()
    return y, phi, dphi, u, r1, n1, n, xo


def _plain_norm_forward(s):
    c = s["case"]
    xo = _plain_norm_parts(s)[-1]
    out = {"x_out": xo.to(_DT[c["res_dtype"]])}
    if c["pre"]:
        r2 = 1 / torch.sqrt((xo * xo).mean(-1, keepdim=True) + EPS)
        out["z"] = (xo * r2 * s["w_pre"]).to(_DT[c["dtype"]])
    return out


def _plain_norm_backward(s):
    c = s["case"]
    y, phi, dphi, u, r1, n1, n, xo = _plain_norm_parts(s)
    out = {}
    dx = s["dx_out"].float()
    if c["pre"]:
        r2 = 1 / torch.sqrt((xo * xo).mean(-1, keepdim=True) + EPS)
        xh = xo * r2
        dz = s["dz"].float()
        out["dw_pre"] = (dz * xh).sum(0)
        t = dz * s["w_pre"]
        dx = dx + r2 * (t - xh * (t * xh).mean(-1, keepdim=True))
    if c["residual"]:
        out["dx"] = dx.to(_DT[c["res_dtype"]])
    if c["scale"]:
        out["dscale"] = (dx * n).sum(0)
    dn = dx * s["scale"] if c["scale"] else dx
    du = dn
    if c["post"]:
        out["dw_post"] = (dn * n1).sum(0)
        t = dn * s["w_post"]
        du = r1 * (t - n1 * (t * n1).mean(-1, keepdim=True))
    out["dy"] = (du * phi if phi is not None else du).to(_DT[c["dtype"]])
    if phi is not None:
        out["dgate"] = (du * y * dphi).to(_DT[c["dtype"]])
    return out


# ------------------------------------------------------------- one pass --
def _own(s):
    from compressed_memory_linear_amd import osr
    c = s["case"]
    op = c["op"]
    if op.startswith("scan"):
        kw = dict(gamma_logit=s["gamma_logit"], y_dtype=_DT[c["y_dtype"]],
                  input_weight={"one": osr.SCAN_ONE, "complement": osr.SCAN_COMPLEMENT,
                                "norm": osr.SCAN_NORM}[c["weight"]])
        if op == "scan_step":
            y, st = osr.lattice_osr_scan_step(s["v"], s["mu_logit"], s["state_in"], y=s["y"],
                                              state_out=s["state_out"], **kw)
            return {"y": y, "state_out": st}
        if op == "scan_prefill":
            y, st = osr.lattice_osr_scan_fwd(s["v"], s["mu_logit"], s["state_in"], lengths=s["lengths"], **kw)
            return {"y": y, "state_out": st}
        y, st, saved = osr.lattice_osr_scan_fwd(s["v"], s["mu_logit"], s["state_in"], lengths=s["lengths"], save=True,
                                                **kw)
        g = osr.lattice_osr_scan_bwd(s["v"], s["mu_logit"], s["dy"], s["dstate_out"], saved=saved,
                                     gamma_logit=s["gamma_logit"], input_weight=kw["input_weight"],
                                     lengths=s["lengths"], grad_dtype=_DT[c["dtype"]])
        return dict(g, y=y, state_out=st)
    kw = dict(gate=s["gate"], gate_kind={"none": osr.GATE_NONE, "gelu": osr.GATE_GELU,
                                         "silu": osr.GATE_SILU}[c["gate"]],
              post_norm=c["post"], w_post=s["w_post"], scale=s["scale"], pre_norm=c["pre"], w_pre=s["w_pre"], eps=EPS)
    if op == "norm_fwd":
        x_out, z = osr.lattice_osr_norm_fwd(s["y"], s["x"], x_dtype=_DT[c["res_dtype"]], **kw)
        return {"x_out": x_out, "z": z} if c["pre"] else {"x_out": x_out}
    return osr.lattice_osr_norm_bwd(s["y"], s["x"], s["dx_out"], s["dz"], grad_dtype=_DT[c["dtype"]], **kw)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("scan_prefill", "scan_step"):
        y, last, _, _ = _plain_scan_forward(state)
        return {"y": y, "state_out": last}
    if op == "scan_train":
        return _plain_scan_train(state)
    return _plain_norm_forward(state) if op == "norm_fwd" else _plain_norm_backward(state)


def work(case):
    """Bytes of the inputs read once and the outputs written once, and the operations of the formulas."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("scan"):
        n, ey = case["B"] * case["T"] * case["D"], 2 if case["y_dtype"] == "bf16" else 4
        tok = 2 + case["gamma"]
        states = 8 * case["B"] * case["D"]
        if case["op"] != "scan_train":
            return {"bytes": n * (e * tok + ey) + states, "flops": n * (12 + 6 * case["gamma"])}
        # the forward's inputs and y; then the backward's inputs (those of the forward again, and dy) and gradients
        return {"bytes": n * (3 * e * tok + 2 * ey) + 2 * states, "flops": n * (40 + 15 * case["gamma"])}
    n, er = case["R"] * case["D"], 2 if case["res_dtype"] == "bf16" else 4
    gated = case["gate"] != "none"
    if case["op"] == "norm_fwd":
        per = e * (1 + gated) + er * (case["residual"] + 1) + e * case["pre"]
        return {"bytes": n * per + 12 * case["D"], "flops": n * (6 + 14 * gated + 6 * case["pre"])}
    per = e * 2 * (1 + gated) + er * (1 + 2 * case["residual"]) + e * case["pre"]
    return {"bytes": n * per + 24 * case["D"], "flops": n * (20 + 30 * gated + 20 * case["pre"])}


# ---------------------------------------------- the definition, in 64 bits --
def exact(case, seed):
    """Token by token from the definition for the recurrence (its gradient by the chain rule, backwards), and
    torch's differentiation of the definition for the norms, in float64."""
    s = prepare(case, seed)
    if case["op"].startswith("scan"):
        return _exact_scan(case, s)
    return _exact_norm(case, s)


def _exact_scan(case, s):
    B, T, D = s["v"].shape
    tm = lambda t: t.double().transpose(0, 1).contiguous()  # time first: one contiguous slice a step
    mu = torch.sigmoid(tm(s["mu_logit"]))
    rest = torch.sigmoid(-tm(s["mu_logit"]))  # 1 - mu, without the cancellation
    v = tm(s["v"])
    gam = torch.sigmoid(tm(s["gamma_logit"])) if case["gamma"] else torch.ones((), dtype=torch.float64,
                                                                              device=v.device)
    if case["weight"] == "one":
        wt = torch.ones_like(mu)
    elif case["weight"] == "complement":
        wt = rest
    else:
        wt = (rest * (2 - rest)).sqrt()
    push = wt * gam * v
    keep = mu
    on = None
    if case["ragged"]:
        on = (torch.arange(T, device=v.device)[:, None] < s["lengths"][None]).unsqueeze(-1)
        keep = mu.masked_fill(~on, 1.0)
        push = push.masked_fill(~on, 0.0)
    H = torch.empty((T + 1, B, D), dtype=torch.float64, device=v.device)
    H[0] = s["state_in"]
    for t in range(T):
        torch.addcmul(push[t], keep[t], H[t], out=H[t + 1])
    back = lambda t: (t if on is None else t.masked_fill(~on, 0.0)).transpose(0, 1).contiguous()
    out = {"y": back(H[1:]), "state_out": H[T].clone()}
    if case["op"] != "scan_train":
        return out
    del push
    dy = tm(s["dy"])
    if on is not None:
        dy = dy.masked_fill(~on, 0.0)
    G = torch.empty((T + 1, B, D), dtype=torch.float64, device=v.device)  # d loss / d h_{t-1}, before y_{t-1}'s share
    G[T] = s["dstate_out"]
    for t in range(T - 1, -1, -1):
        torch.mul(torch.add(G[t + 1], dy[t], out=dy[t]), keep[t], out=G[t])
    dh = dy  # now d loss / d h_t
    slope = mu * rest
    turn = dh * H[:T] * slope
    if case["weight"] == "complement":
        turn -= dh * gam * v * slope
    elif case["weight"] == "norm":
        turn -= dh * gam * v * mu * slope / wt.clamp_min(1e-300)
    out["dmu_logit"] = back(turn)
    out["dv"] = back(dh * wt * gam)
    if case["gamma"]:
        out["dgamma_logit"] = back(dh * wt * v * gam * (1 - gam))
    out["dstate_in"] = G[0].clone()
    return out


def _exact_norm(case, s):
    D = case["D"]
    leaf = {k: s[k].double().requires_grad_(case["op"] == "norm_bwd")
            for k in ("y", "gate", "x", "w_post", "scale", "w_pre") if s[k] is not None}
    m = leaf["y"]
    if case["gate"] == "gelu":
        m = m * (leaf["gate"] * torch.special.ndtr(leaf["gate"]))
    elif case["gate"] == "silu":
        m = m * (leaf["gate"] * torch.sigmoid(leaf["gate"]))
    if case["post"]:
        m = m * (m.square().sum(-1, keepdim=True) / D + EPS).rsqrt() * leaf["w_post"]
    if case["scale"]:
        m = m * leaf["scale"]
    if case["residual"]:
        m = leaf["x"] + m
    z = m * (m.square().sum(-1, keepdim=True) / D + EPS).rsqrt() * leaf["w_pre"] if case["pre"] else None
    if case["op"] == "norm_fwd":
        return {"x_out": m, "z": z} if case["pre"] else {"x_out": m}
    loss = (m * s["dx_out"].double()).sum()
    if z is not None:
        loss = loss + (z * s["dz"].double()).sum()
    names = list(leaf)
    grads = torch.autograd.grad(loss, [leaf[k] for k in names])
    return {"d" + k: g for k, g in zip(names, grads)}
