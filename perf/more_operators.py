"""What is timed of the selective state space layer: its scan, the short
causal convolution in front of it and the layer norm around it; the cases,
their inputs, one pass through each and its exact result.

    ssm    per channel c and state n, with delta = softplus(dt + dt_bias):
           h_t = exp(delta_t A[c,n]) h_{t-1} + delta_t x_t B_t[n],
           y_t = (sum_n C_t[n] h_t[n] + D[c] x_t) z_t sigmoid(z_t)
    conv   p_t = bias[c] + sum_j w[c,j] x_{t-W+1+j},  y_t = p_t sigmoid(p_t)
    ln     x' = x + y,  z = (x' - mean(x')) / sqrt(var(x') + eps) w + b over a row

``own`` chooses between the plain form (elementary torch operations in 32 bits)
and the calls of this package.
"""
import math

import torch

own = False

EPS = 1e-5
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases --
def _ssm(name, op, B, T, D, N, dtype="bf16", G=1, **kw):
    return {"name": name, "op": op, "B": B, "T": T, "D": D, "N": N, "G": G, "dtype": dtype, "y_dtype": dtype,
            "skip": True, "gate": True, "bias": True, "ragged": False, "packed": False, "slices": True, **kw}


def _conv(name, op, B, T, D, W=4, dtype="bf16", **kw):
    return {"name": name, "op": op, "B": B, "T": T, "D": D, "W": W, "dtype": dtype, "bias": True, "silu": True,
            "ragged": False, "packed": False, "slices": True, **kw}


def listed():
    return [
        # one layer's prefill over eight sequences of 4096 tokens, 2048 channels of 16 states: the ordinary call; the
        # gate is the second half of the layer's one input projection, B and C are slices of another
        _ssm("ssm_prefill_b8_t4096_d2048", "ssm_prefill", 8, 4096, 2048, 16),
        # one long document: few channels for the chip, so the time axis has to fill it; the largest call
        _ssm("ssm_prefill_b1_t65536_d2048", "ssm_prefill", 1, 65536, 2048, 16),
        # a padded batch of prompts of different lengths (one empty, one of a single token), odd sizes, fp32, no gate
        _ssm("ssm_prefill_padded_b7_t1531", "ssm_prefill", 7, 1531, 1001, 13, "f32", ragged=True, gate=False,
             slices=False),
        # a training step, documents packed behind one another in each row: forward and all gradients
        _ssm("ssm_train_b4_t4096_d2048", "ssm_train", 4, 4096, 2048, 16, packed=True),
        # a small fp32 training step with a wide state and two groups of B and C, as when a model is tried out
        _ssm("ssm_train_b3_t777_d514_n64", "ssm_train", 3, 777, 514, 64, "f32", G=2, slices=False),
        # one new token for each of 256 sequences, 32 heads of 128: the serving step of a full batch
        _ssm("ssm_step_b256_d4096", "ssm_step", 256, 1, 4096, 16),
        # the convolution in front of the first case: its input is the first half of the input projection
        _conv("conv_prefill_b8_t4096_d2048", "conv_prefill", 8, 4096, 2048),
        # the convolution's training step on packed documents, whose taps stop at their borders
        _conv("conv_train_b8_t4096_d2048", "conv_train", 8, 4096, 2048, packed=True),
        # one new token for one sequence: the smallest call, where only latency counts
        _conv("conv_step_b1_d2048", "conv_step", 1, 1, 2048, slices=False),
        # between two layers in training or prefill: the residual and the norm before the next layer
        {"name": "ln_fwd_r32768_d2048", "op": "ln_fwd", "R": 32768, "D": 2048, "dtype": "bf16", "res_dtype": "bf16",
         "residual": True, "affine": True},
        # its backward, with the sums over all rows for the weight's and the bias's gradient
        {"name": "ln_bwd_r32768_d2048", "op": "ln_bwd", "R": 32768, "D": 2048, "dtype": "bf16", "res_dtype": "bf16",
         "residual": True, "affine": True},
        # the backward at odd sizes, activations in bf16 beside a residual stream in fp32
        {"name": "ln_bwd_r2331_d1001", "op": "ln_bwd", "R": 2331, "D": 1001, "dtype": "bf16", "res_dtype": "f32",
         "residual": True, "affine": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    kind = rng.choice(["ssm", "ssm", "conv", "ln"])
    if kind == "ln":
        D = _log_int(rng, 16, 8192)
        if rng.random() < 0.6:
            D = max(16, D // 16 * 16)
        R = _log_int(rng, 1, max(1, min(100_000, 24_000_000 // D)))
        return {"op": rng.choice(["ln_fwd", "ln_bwd"]), "R": R, "D": D, "dtype": dtype,
                "res_dtype": rng.choice([dtype, "f32"]), "residual": rng.random() < 0.7,
                "affine": rng.random() < 0.8}
    step = rng.random() < 0.25
    B = _log_int(rng, 1, 512 if step else 32)
    T = 1 if step else _log_int(rng, 1, 65536)
    D = _log_int(rng, 16, 8192)
    if rng.random() < 0.6:
        D = max(16, D // 16 * 16)
    N = rng.choice([1, 4, 8, 16, 16, 16, 32, 64, rng.randint(1, 64)])
    # values of the state (ssm) or of one tensor (conv): well under the largest listed case
    most = 24_000_000 if kind == "conv" or step else 400_000_000 // max(N, 16)
    while B * T * D > most:
        if B > 1 and rng.random() < 0.5:
            B = (B + 1) // 2
        elif T > 1:
            T = (T + 1) // 2
        else:
            D = (D + 1) // 2
    op = kind + "_" + ("step" if step else rng.choice(["prefill", "train"]))
    ragged, packed = not step and rng.random() < 0.3, not step and rng.random() < 0.3
    if kind == "conv":
        c = _conv("", op, B, T, D, rng.choice([2, 3, 4, 4, 4]), dtype, bias=rng.random() < 0.7, silu=rng.random() < 0.8,
                  ragged=ragged, packed=packed, slices=not step and rng.random() < 0.5)
    else:
        G = rng.choice([g for g in (1, 1, 1, 2, 4) if D % g == 0])
        c = _ssm("", op, B, T, D, N, dtype, G, y_dtype=rng.choice([dtype, "f32"]), skip=rng.random() < 0.8,
                 gate=rng.random() < 0.7, bias=rng.random() < 0.7, ragged=ragged, packed=packed,
                 slices=rng.random() < 0.5)
    del c["name"]
    return c


# --------------------------------------------------------------- inputs --
def prepare(case, seed):
    """Activations of unit size; decays -1 .. -N with some spread, steps delta spread over 0.001 .. 0.1 by
    their bias, as a trained layer has them; norm weights around 1.  Everything from the seed alone."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = _DT[case["dtype"]]
    f32 = torch.float32

    def normal(*shape, mean=0.0, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dtype)

    s = {"case": dict(case)}
    if case["op"].startswith("ln"):
        R, D = case["R"], case["D"]
        rt = _DT[case["res_dtype"]]
        s["x"] = normal(R, D, mean=0.5, std=2.0, dtype=rt)
        s["y"] = normal(R, D) if case["residual"] else None
        s["w"] = normal(D, mean=1.0, std=0.2, dtype=f32) if case["affine"] else None
        s["b"] = normal(D, std=0.2, dtype=f32) if case["affine"] else None
        if case["op"] == "ln_bwd":
            s["dx_out"] = normal(R, D, dtype=rt) if case["residual"] else None
            s["dz"] = normal(R, D)
        return s
    B, T, D = case["B"], case["T"], case["D"]
    s["lengths"] = s["segments"] = None
    if case["ragged"]:
        n = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        if B >= 3:
            n[0], n[1], n[2] = 0, 1, T
        s["lengths"] = n
    if case["packed"]:  # document numbers, a few borders in every row
        s["segments"] = (torch.rand((B, T), generator=g, device=dev) < 4.0 / max(T, 4)).cumsum(1).to(torch.int32)
    step = case["op"].endswith("step")
    if case["op"].startswith("conv"):
        W = case["W"]
        s["x"] = normal(B, T, 2 * D)[..., :D] if case["slices"] else normal(B, T, D)
        s["w"] = normal(D, W, std=0.4, dtype=f32)
        s["bias"] = normal(D, std=0.2, dtype=f32) if case["bias"] else None
        s["hist"] = normal(B, W - 1, D)
        if case["op"] == "conv_train":
            s["dy"] = normal(B, T, D)
            s["dhist_out"] = normal(B, W - 1, D)
        if step:  # a serving loop keeps its output buffers
            s["out"] = torch.empty((B, T, D), dtype=dt, device=dev)
            s["hist_out"] = torch.empty_like(s["hist"])
        return s
    N, G = case["N"], case["G"]
    yt = _DT[case["y_dtype"]]
    s["x"] = normal(B, T, D)
    first = torch.exp(torch.rand((D,), generator=g, device=dev) * math.log(100.0) + math.log(1e-3))
    bias = first + torch.log(-torch.expm1(-first))  # softplus(bias) = first
    s["dt"] = normal(B, T, D, std=0.5, mean=0.0 if case["bias"] else -4.0)
    s["dt_bias"] = bias if case["bias"] else None
    s["A"] = -torch.arange(1, N + 1, device=dev, dtype=f32) * torch.exp(normal(D, N, std=0.1, dtype=f32))
    if case["slices"]:
        proj = normal(B, T, 2 * G * N + 64)
        s["Bm"] = proj[..., 64:64 + G * N].unflatten(-1, (G, N))
        s["Cm"] = proj[..., 64 + G * N:].unflatten(-1, (G, N))
    else:
        s["Bm"], s["Cm"] = normal(B, T, G, N), normal(B, T, G, N)
    s["D"] = normal(D, mean=1.0, std=0.2, dtype=f32) if case["skip"] else None
    s["z"] = None
    if case["gate"]:
        s["z"] = normal(B, T, 2 * D)[..., D:] if case["slices"] else normal(B, T, D)
    s["state_in"] = normal(B, D, N, dtype=f32)
    if case["op"] == "ssm_train":
        s["dy"] = normal(B, T, D, dtype=yt)
        s["dstate_out"] = normal(B, D, N, dtype=f32)
    if step:
        s["out"] = torch.empty((B, T, D), dtype=yt, device=dev)
        s["state_out"] = torch.empty((B, D, N), device=dev)
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


def _plain_masks(s):
    """[B,T] truth values: tokens that are no padding, and tokens whose document began with them (None: all, none)."""
    B, T = s["x"].shape[:2]
    ok = cut = None
    if s["lengths"] is not None:
        ok = torch.arange(T, device=s["x"].device)[None] < s["lengths"][:, None]
    if s["segments"] is not None:
        cut = torch.zeros((B, T), dtype=torch.bool, device=s["x"].device)
        cut[:, 1:] = s["segments"][:, 1:] != s["segments"][:, :-1]
    return ok, cut


def _plain_ssm_parts(s):
    c = s["case"]
    B, T, D = s["x"].shape
    G, N = c["G"], c["N"]
    ok, cut = _plain_masks(s)
    raw = s["dt"].float()
    if s["dt_bias"] is not None:
        raw = raw + s["dt_bias"]
    delta = raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs()))
    if ok is not None:  # a padded token keeps the state
        delta = torch.where(ok[..., None], delta, 0.0)
    x = s["x"].float()
    u = delta * x
    wide = lambda m: m.float().unsqueeze(3).expand(B, T, G, D // G, N).reshape(B, T, D, N)
    Bw, Cw = wide(s["Bm"]), wide(s["Cm"])
    a = torch.exp(delta[..., None] * s["A"])
    if cut is not None:
        a = torch.where((cut & ok if ok is not None else cut)[..., None, None], 0.0, a)
    first = u[..., None] * Bw
    first[:, 0] += a[:, 0] * s["state_in"]
    h = _plain_linear_scan(a, first)
    del first
    core = (h * Cw).sum(-1)
    if s["D"] is not None:
        core = core + s["D"] * x
    return ok, raw, delta, x, u, Bw, Cw, a, h, core


def _masked(ok, t):
    return t if ok is None else torch.where(ok[(...,) + (None,) * (t.dim() - 2)], t, 0.0)


def _plain_gate(s):
    if s["z"] is None:
        return None, None
    z = s["z"].float()
    sg = 1 / (1 + torch.exp(-z))
    return z * sg, sg * (1 + z * (1 - sg))


def _plain_ssm_forward(s):
    ok, *_, h, core = _plain_ssm_parts(s)
    phi, _ = _plain_gate(s)
    y = core if phi is None else core * phi
    return {"y": _masked(ok, y).to(_DT[s["case"]["y_dtype"]]), "state_out": h[:, -1].clone()}


def _plain_ssm_train(s):
    c = s["case"]
    dt = _DT[c["dtype"]]
    G, N, D = c["G"], c["N"], c["D"]
    ok, raw, delta, x, u, Bw, Cw, a, h, core = _plain_ssm_parts(s)
    phi, dphi = _plain_gate(s)
    out = {"y": _masked(ok, core if phi is None else core * phi).to(_DT[c["y_dtype"]]), "state_out": h[:, -1].clone()}
    dy = _masked(ok, s["dy"].float())
    if phi is not None:
        out["dz"] = (dy * core * dphi).to(dt)
        dy = dy * phi
    del core
    narrow = lambda t: t.unflatten(2, (G, D // G)).sum(3).to(dt)
    out["dC"] = narrow(dy[..., None] * h)
    push = dy[..., None] * Cw
    del Cw
    push[:, -1] += s["dstate_out"]
    nxt = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    lam = _plain_linear_scan(nxt.flip(1), push.flip(1)).flip(1)
    del nxt, push
    out["dB"] = narrow(lam * u[..., None])
    du = _masked(ok, (lam * Bw).sum(-1))
    del Bw
    out["dstate_in"] = a[:, 0] * lam[:, 0]
    lam *= a
    lam[:, 1:] *= h[:, :-1]
    lam[:, 0] *= s["state_in"]
    ddelta = _masked(ok, (lam * s["A"]).sum(-1)) + du * x
    out["dA"] = (lam * delta[..., None]).sum((0, 1))
    ddt = ddelta / (1 + torch.exp(-raw))
    out["ddt"] = ddt.to(dt)
    if s["dt_bias"] is not None:
        out["ddt_bias"] = ddt.sum((0, 1))
    dx = du * delta
    if s["D"] is not None:
        dx = dx + dy * s["D"]
        out["dD"] = (dy * x).sum((0, 1))
    out["dx"] = dx.to(dt)
    return out


def _plain_conv_parts(s):
    """The taps' inputs [W,B,T,D] (zero past a border), the sum and the history behind the last token."""
    W = s["case"]["W"]
    B, T, D = s["x"].shape
    ok, cut = _plain_masks(s)
    x = s["x"].float()
    if ok is not None:
        x = torch.where(ok[..., None], x, 0.0)
    rows = torch.cat([s["hist"].float(), x], 1)  # row t + W - 1 is token t
    seg = torch.zeros((B, T + W - 1), dtype=torch.int64, device=x.device)
    if s["segments"] is not None:
        seg[:, W - 1:] = s["segments"]
        seg[:, :W - 1] = s["segments"][:, :1]
    # documents are numbered upwards, so one that differs from the token's own lies before its border
    reach = lambda j: (seg[:, j:j + T] == seg[:, W - 1:])[..., None]
    taps = torch.stack([torch.where(reach(j), rows[:, j:j + T], 0.0) for j in range(W)])
    pre = (taps * s["w"].t()[:, None, None]).sum(0)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    n = torch.full((B,), T, device=x.device) if s["lengths"] is None else s["lengths"].long()
    at = n[:, None] + torch.arange(W - 1, device=x.device)  # rows of the history behind the last token
    same = torch.gather(seg, 1, at) == torch.gather(seg, 1, (n + W - 2)[:, None])
    tail = torch.where(same[..., None], torch.gather(rows, 1, at[..., None].expand(-1, -1, D)), 0.0)
    return ok, taps, pre, reach, at, same, tail


def _plain_act(c, p):
    if not c["silu"]:
        return p, torch.ones_like(p)
    sg = 1 / (1 + torch.exp(-p))
    return p * sg, sg * (1 + p * (1 - sg))


def _plain_conv_forward(s):
    dt = _DT[s["case"]["dtype"]]
    ok, _, pre, _, _, _, tail = _plain_conv_parts(s)
    return {"y": _masked(ok, _plain_act(s["case"], pre)[0]).to(dt), "hist_out": tail.to(dt)}


def _plain_conv_train(s):
    c = s["case"]
    dt, W = _DT[c["dtype"]], c["W"]
    B, T, D = s["x"].shape
    ok, taps, pre, reach, at, same, tail = _plain_conv_parts(s)
    act, slope = _plain_act(c, pre)
    out = {"y": _masked(ok, act).to(dt), "hist_out": tail.to(dt)}
    dp = _masked(ok, s["dy"].float() * slope)
    drows = torch.zeros((B, T + W - 1, D), device=dp.device)
    for j in range(W):
        drows[:, j:j + T] += torch.where(reach(j), dp * s["w"][:, j], 0.0)
    back = torch.where(same[..., None], s["dhist_out"].float(), 0.0)
    drows.scatter_add_(1, at[..., None].expand(-1, -1, D), back)
    out["dx"] = _masked(ok, drows[:, W - 1:]).to(dt)
    out["dhist_in"] = drows[:, :W - 1].to(dt)
    out["dw"] = (taps * dp).sum((1, 2)).t().contiguous()
    if s["bias"] is not None:
        out["dbias"] = dp.sum((0, 1))
    return out


def _plain_ln(s):
    c = s["case"]
    dt, rt = _DT[c["dtype"]], _DT[c["res_dtype"]]
    x = s["x"].float()
    if c["residual"]:
        x = x + s["y"].float()
    mid = x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((mid * mid).mean(-1, keepdim=True) + EPS)
    n = mid * r
    if c["op"] == "ln_fwd":
        z = n * s["w"] + s["b"] if c["affine"] else n
        return {"z": z.to(dt), "x_out": x.to(rt)} if c["residual"] else {"z": z.to(dt)}
    dz = s["dz"].float()
    t = dz * s["w"] if c["affine"] else dz
    dx = r * (t - t.mean(-1, keepdim=True) - n * (t * n).mean(-1, keepdim=True))
    if s["dx_out"] is not None:
        dx = dx + s["dx_out"].float()
    out = {"dx": dx.to(rt)}
    if c["residual"] and dt != rt:
        out["dy"] = dx.to(dt)
    if c["affine"]:
        out["dw"], out["db"] = (dz * n).sum(0), dz.sum(0)
    return out


# ------------------------------------------------------------- one pass --
def _own(s):
    from compressed_memory_linear_amd import osr
    c = s["case"]
    op, dt = c["op"], _DT[c["dtype"]]
    if op == "ln_fwd":
        x_out, z = osr.lattice_osr_layernorm_fwd(s["x"], s["y"], w=s["w"], b=s["b"], eps=EPS, z_dtype=dt)
        return {"z": z, "x_out": x_out} if c["residual"] else {"z": z}
    if op == "ln_bwd":
        g = osr.lattice_osr_layernorm_bwd(s["x"], s["y"], s["dx_out"], s["dz"], w=s["w"], b=s["b"], eps=EPS,
                                          grad_dtype=dt)
        return {k: t for k, t in g.items() if k != "dy" or _DT[c["res_dtype"]] != dt}
    if op.startswith("conv"):
        kw = dict(act=osr.CONV_SILU if c["silu"] else osr.CONV_NONE)
        if op == "conv_step":
            y, hist = osr.lattice_osr_conv_step(s["x"], s["w"], s["hist"], s["bias"], y=s["out"],
                                                hist_out=s["hist_out"], **kw)
            return {"y": y, "hist_out": hist}
        kw.update(lengths=s["lengths"], segments=s["segments"])
        y, hist = osr.lattice_osr_conv_fwd(s["x"], s["w"], s["bias"], s["hist"], return_history=True, **kw)
        if op == "conv_prefill":
            return {"y": y, "hist_out": hist}
        g = osr.lattice_osr_conv_bwd(s["x"], s["w"], s["dy"], s["bias"], s["hist"], s["dhist_out"], grad_dtype=dt, **kw)
        return dict(g, y=y, hist_out=hist)
    args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
    kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    yt = _DT[c["y_dtype"]]
    if op == "ssm_step":
        y, st = osr.lattice_osr_ssm_step(*args, s["state_in"], y_dtype=yt, y=s["out"], state_out=s["state_out"], **kw)
        return {"y": y, "state_out": st}
    kw.update(lengths=s["lengths"], segments=s["segments"])
    if op == "ssm_prefill":
        y, st = osr.lattice_osr_ssm_fwd(*args, s["state_in"], y_dtype=yt, **kw)
        return {"y": y, "state_out": st}
    y, st, saved = osr.lattice_osr_ssm_fwd(*args, s["state_in"], y_dtype=yt, save=True, **kw)
    g = osr.lattice_osr_ssm_bwd(*args, s["dy"], s["dstate_out"], saved=saved, grad_dtype=dt, **kw)
    return dict(g, y=y, state_out=st)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op.startswith("ln"):
        return _plain_ln(state)
    if op.startswith("conv"):
        return _plain_conv_train(state) if op == "conv_train" else _plain_conv_forward(state)
    return _plain_ssm_train(state) if op == "ssm_train" else _plain_ssm_forward(state)


def work(case):
    """Bytes of the inputs read once and the outputs written once (a training step's backward reads the forward's
    inputs again), and the operations of the formulas."""
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"].startswith("ln"):
        n, er, two = c["R"] * c["D"], 2 if c["res_dtype"] == "bf16" else 4, c["residual"]
        if c["op"] == "ln_fwd":
            return {"bytes": n * (er * (1 + two) + e * (1 + two)) + 8 * c["D"] * c["affine"], "flops": n * (7 + two)}
        also = two and er != e
        return {"bytes": n * (er * (2 + two) + e * (1 + two + also)) + 12 * c["D"] * c["affine"], "flops": n * 18}
    n, rows = c["B"] * c["T"] * c["D"], c["B"] * c["T"]
    if c["op"].startswith("conv"):
        small = 2 * c["B"] * (c["W"] - 1) * c["D"] * e + 4 * c["D"] * (c["W"] + c["bias"])
        flops = n * (2 * c["W"] + 6 * c["silu"])
        if c["op"] != "conv_train":
            return {"bytes": n * 2 * e + small, "flops": flops}
        return {"bytes": n * 5 * e + 3 * small, "flops": flops * 2 + n * (4 * c["W"] + 8 * c["silu"])}
    ey, N = 2 if c["y_dtype"] == "bf16" else 4, c["N"]
    bc = rows * 2 * c["G"] * N * e
    states = 8 * c["B"] * c["D"] * N
    weights = 4 * c["D"] * (N + c["skip"] + c["bias"])
    fwd = n * (e * (2 + c["gate"]) + ey) + bc + states + weights
    if c["op"] != "ssm_train":
        return {"bytes": fwd, "flops": n * (7 * N + 14)}
    back = n * (e * 2 * (2 + c["gate"]) + ey) + 2 * bc + states + 2 * weights
    return {"bytes": fwd + back, "flops": n * (7 * N + 14 + 20 * N + 40)}


# ---------------------------------------------- the definition, in 64 bits --
def exact(case, seed):
    """Token by token from the definition for the recurrence (its gradient by the chain rule, backwards), and
    torch's differentiation of the definitions for the convolution and the norm, in float64."""
    s = prepare(case, seed)
    if case["op"].startswith("ln"):
        return _exact_ln(case, s)
    if case["op"].startswith("conv"):
        return _exact_conv(case, s)
    return _exact_ssm(case, s)


def _exact_ssm(case, s):
    B, T, D = s["x"].shape
    G, N = case["G"], case["N"]
    train = case["op"] == "ssm_train"
    dev = s["x"].device
    tm = lambda t: t.transpose(0, 1)  # time first
    on = torch.ones((T, B, 1), device=dev, dtype=torch.float64)
    keep = torch.ones((T, B, 1), device=dev, dtype=torch.float64)
    if case["ragged"]:
        on = (torch.arange(T, device=dev)[:, None] < s["lengths"][None]).double().unsqueeze(-1)
    if case["packed"]:
        seg = tm(s["segments"])
        keep[1:, :, 0] = (seg[1:] == seg[:-1]).double()
        keep = torch.where(on > 0, keep, 1.0)
    raw = tm(s["dt"]).double()
    if case["bias"]:
        raw = raw + s["dt_bias"].double()
    delta = torch.logaddexp(raw, torch.zeros((), dtype=torch.float64, device=dev)) * on
    x = tm(s["x"]).double()
    u = delta * x
    A = s["A"].double().view(G, D // G, N)
    Bm, Cm = tm(s["Bm"]), tm(s["Cm"])  # [T,B,G,N]
    view = lambda t: t.reshape(t.shape[:-1] + (G, D // G))
    dv, uv, kv = view(delta), view(u), keep.view(T, B, 1, 1, 1)
    at = lambda m, t: m[t].double().unsqueeze(2)  # [B,G,1,N]
    h = s["state_in"].double().view(B, G, D // G, N)
    H = torch.empty((T + 1, B, G, D // G, N), dtype=torch.float64, device=dev) if train else None
    core = torch.empty((T, B, D), dtype=torch.float64, device=dev)
    for t in range(T):
        if train:
            H[t] = h
        h = torch.exp(dv[t].unsqueeze(-1) * A) * (h * kv[t]) + uv[t].unsqueeze(-1) * at(Bm, t)
        core[t] = (h * at(Cm, t)).sum(-1).view(B, D)
    if case["skip"]:
        core += s["D"].double() * x
    if case["gate"]:
        z = tm(s["z"]).double()
        sg = torch.sigmoid(z)
    y = core * z * sg if case["gate"] else core
    back = lambda t: tm(t * on).contiguous()
    out = {"y": back(y), "state_out": h.reshape(B, D, N).clone()}
    if not train:
        return out
    H[T] = h
    dy = tm(s["dy"]).double() * on
    if case["gate"]:
        out["dz"] = back(dy * core * (sg + z * sg * (1 - sg)))
        dy = dy * z * sg
    dyv = view(dy)
    lam = s["dstate_out"].double().view(B, G, D // G, N).clone()
    dA = torch.zeros((G, D // G, N), dtype=torch.float64, device=dev)
    du, dd = torch.empty_like(uv), torch.empty_like(uv)
    dB, dC = (torch.empty((T, B, G, N), dtype=torch.float64, device=dev) for _ in range(2))
    for t in range(T - 1, -1, -1):
        lam = lam + dyv[t].unsqueeze(-1) * at(Cm, t)
        dC[t] = (dyv[t].unsqueeze(-1) * H[t + 1]).sum(2)
        dB[t] = (lam * uv[t].unsqueeze(-1)).sum(2)
        du[t] = (lam * at(Bm, t)).sum(-1)
        lam = lam * torch.exp(dv[t].unsqueeze(-1) * A) * kv[t]
        p = lam * H[t]
        dd[t] = (p * A).sum(-1)
        dA += (p * dv[t].unsqueeze(-1)).sum(0)
    du, dd = du.reshape(T, B, D) * on, dd.reshape(T, B, D) * on
    ddt = (dd + du * x) * torch.sigmoid(raw)
    dx = du * delta
    if case["skip"]:
        dx = dx + dy * s["D"].double()
        out["dD"] = (dy * x).sum((0, 1))
    if case["bias"]:
        out["ddt_bias"] = ddt.sum((0, 1))
    out.update(dx=back(dx), ddt=back(ddt), dA=dA.view(D, N), dB=tm(dB).contiguous(), dC=tm(dC).contiguous(),
               dstate_in=lam.reshape(B, D, N).clone())
    return out


def _exact_conv(case, s):
    B, T, D = s["x"].shape
    W = case["W"]
    dev = s["x"].device
    train = case["op"] == "conv_train"
    leaf = {k: s[n].double().requires_grad_(train) for k, n in (("x", "x"), ("w", "w"), ("bias", "bias"),
                                                              ("hist_in", "hist")) if s[n] is not None}
    n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    ids = None if s["segments"] is None else s["segments"]
    seqs, tails = [], []
    for b in range(B):  # one sequence at a time, its documents as filters over the rows they own
        rows = torch.cat([leaf["hist_in"][b], leaf["x"][b, :n[b]]])
        own_id = torch.zeros(len(rows), dtype=torch.int64, device=dev)
        if ids is not None:
            own_id[:W - 1] = ids[b, 0]
            own_id[W - 1:] = ids[b, :n[b]]
        acc = torch.zeros((n[b], D), dtype=torch.float64, device=dev)
        for back in range(W):  # the row `back` tokens before each
            r = rows[W - 1 - back:W - 1 - back + n[b]]
            same = own_id[W - 1 - back:W - 1 - back + n[b]] == own_id[W - 1:]
            acc = acc + r * same[:, None] * leaf["w"][:, W - 1 - back]
        if case["bias"]:
            acc = acc + leaf["bias"]
        if case["silu"]:
            acc = torch.nn.functional.silu(acc)
        seqs.append(torch.cat([acc, acc.new_zeros((T - n[b], D))]))
        tails.append(rows[n[b]:] * (own_id[n[b]:] == own_id[-1])[:, None])
    y, tail = torch.stack(seqs), torch.stack(tails)
    out = {"y": y.detach(), "hist_out": tail.detach()}
    if train:
        loss = (y * s["dy"].double()).sum() + (tail * s["dhist_out"].double()).sum()
        out.update({"d" + k: g for k, g in zip(leaf, torch.autograd.grad(loss, list(leaf.values())))})
    return out


def _exact_ln(case, s):
    D = case["D"]
    back = case["op"] == "ln_bwd"
    leaf = {k: s[k].double().requires_grad_(back) for k in ("x", "w", "b") if s[k] is not None}
    x = leaf["x"]
    if case["residual"]:
        x = x + s["y"].double()
    mean = x.sum(-1, keepdim=True) / D
    z = (x - mean) * (((x - mean) ** 2).sum(-1, keepdim=True) / D + EPS).rsqrt()
    if case["affine"]:
        z = z * leaf["w"] + leaf["b"]
    if not back:
        return {"z": z, "x_out": x} if case["residual"] else {"z": z}
    loss = (z * s["dz"].double()).sum()
    if s["dx_out"] is not None:
        loss = loss + (x * s["dx_out"].double()).sum()
    out = {"d" + k: g for k, g in zip(leaf, torch.autograd.grad(loss, list(leaf.values())))}
    if case["residual"] and case["dtype"] != case["res_dtype"]:
        out["dy"] = out["dx"].clone()
    return out
