"""Host-only checks of the state space layer's operators (lattice_osr_conv_*,
lattice_osr_ssm_*, lattice_osr_layernorm_*): argument checks of the C ABI with
the documented status codes, before any HIP call, and of the Python binding (no
GPU needed)."""
import ctypes
import math

import pytest
import torch

from compressed_memory_linear_amd import osr

# Fake device addresses: only compared and range-checked on the host, because
# every case below fails validation first.
BASE, GAP = 1 << 40, 1 << 34
WS = BASE + 60 * GAP
BIG = 1 << 33


def _fake(names):
    return {n: BASE + i * GAP for i, n in enumerate(names)}


def _call(fn, desc, names, p, tail=()):
    """The C entry fn with the pointers p by name; tail: what follows a name, by name."""
    args = []
    for n in names:
        args.append(p[n])
        args += dict(tail).get(n, [])
    return getattr(osr.load_library(), "lattice_osr_" + fn)(ctypes.byref(desc) if desc is not None else None, *args, None)


CF = ("x", "w", "bias", "lengths", "segments", "hist_in", "hist_out", "y")
CB = ("x", "w", "bias", "lengths", "segments", "hist_in", "dy", "dhist_out", "dx", "dw", "dbias", "dhist_in", "ws")
CS = ("x", "w", "bias", "hist_in", "hist_out", "y")
SF = ("x", "dt", "A", "Bm", "Cm", "skip", "z", "dt_bias", "lengths", "segments", "state_in", "state_out", "y", "saved", "ws")
SB = ("x", "dt", "A", "Bm", "Cm", "skip", "z", "dt_bias", "lengths", "segments", "saved", "dy", "dstate_out", "dx", "ddt",
      "dA", "dB", "dC", "dskip", "dz", "ddt_bias", "dstate_in", "ws")
SS = ("x", "dt", "A", "Bm", "Cm", "skip", "z", "dt_bias", "state_in", "state_out", "y")
LF = ("x", "y", "w", "b", "x_out", "z")
LB = ("x", "y", "w", "dx_out", "dz", "dx", "dy", "dw", "db", "ws")
NAMES = dict(conv_fwd=CF, conv_bwd=CB, conv_step=CS, ssm_fwd=SF, ssm_bwd=SB, ssm_step=SS, layernorm_fwd=LF,
             layernorm_bwd=LB)
OUTS = dict(conv_fwd=("hist_out", "y"), conv_bwd=("dx", "dw", "dbias", "dhist_in", "ws"), conv_step=("hist_out", "y"),
            ssm_fwd=("state_out", "y", "saved"), ssm_bwd=SB[13:], ssm_step=("state_out", "y"), layernorm_fwd=("x_out", "z"),
            layernorm_bwd=("dx", "dy", "dw", "db", "ws"))
# outputs that may be an input itself (not with an overlap in part)
SAME = {("conv_step", "hist_out", "hist_in"), ("ssm_fwd", "state_out", "state_in"), ("ssm_step", "state_out", "state_in"),
        ("layernorm_fwd", "x_out", "x"), ("layernorm_bwd", "dx", "dx_out")}


def call(fn, desc, p, saved=BIG, ws=BIG):
    return _call(fn, desc, NAMES[fn], {**p, "ws": p.get("ws", WS)}, {"saved": [saved], "ws": [ws]})


def desc_of(fn, **kw):
    if fn.startswith("conv"):
        return osr.make_conv_desc(**{**dict(B=2, T=1, D=64, W=4), **kw})
    if fn.startswith("ssm"):
        return osr.make_ssm_desc(**{**dict(B=2, T=1, D=64, N=16, G=2), **kw})
    return osr.make_layernorm_desc(**{**dict(R=4, D=64), **kw})


def fakes(fn):
    return _fake([n for n in NAMES[fn] if n != "ws"])


def names_of(fn, desc):
    """The pointers that a call takes: the forward scan's workspace where it has one."""
    none = fn == "ssm_fwd" and osr.lattice_osr_ssm_workspace_bytes(desc) == 0
    return [n for n in NAMES[fn] if not (none and n == "ws")]


SHAPE, NO, NULL = osr.ERR_SHAPE, osr.ERR_UNSUPPORTED, osr.ERR_NULL
CONV_BAD = [("B", 0, SHAPE), ("T", 0, SHAPE), ("D", -1, SHAPE), ("D", (1 << 20) + 1, SHAPE), ("T", (1 << 30) + 1, SHAPE),
            ("W", 0, NO), ("W", 9, NO), ("act", 2, NO), ("act", -1, NO), ("in_dtype", 2, NO), ("y_dtype", -1, NO),
            ("grad_dtype", 7, NO), ("x_row", 63, SHAPE), ("x_row", -64, SHAPE), ("x_row", (1 << 22) + 1, SHAPE),
            ("B", 1 << 25, SHAPE)]
SSM_BAD = [("B", 0, SHAPE), ("T", -2, SHAPE), ("D", 0, SHAPE), ("D", (1 << 20) + 2, SHAPE), ("N", 0, NO), ("N", 65, NO),
           ("G", 0, SHAPE), ("G", 3, SHAPE), ("G", -2, SHAPE), ("in_dtype", 3, NO), ("y_dtype", 2, NO), ("grad_dtype", -1, NO),
           ("softplus", 2, NO), ("x_row", 1, SHAPE), ("dt_row", 63, SHAPE), ("z_row", -1, SHAPE), ("b_row", 31, SHAPE),
           ("c_row", 5, SHAPE), ("b_row", (1 << 22) + 1, SHAPE), ("B", 1 << 21, SHAPE)]
LN_BAD = [("R", 0, SHAPE), ("D", 0, SHAPE), ("D", 16385, NO), ("in_dtype", 2, NO), ("res_dtype", 2, NO), ("grad_dtype", 2, NO),
          ("eps", 0.0, NO), ("eps", -1.0, NO), ("eps", math.nan, NO), ("eps", math.inf, NO), ("eps", 1e-39, NO)]


@pytest.mark.parametrize("kind,field,value,status", [("conv", *c) for c in CONV_BAD] + [("ssm", *c) for c in SSM_BAD] +
                         [("layernorm", *c) for c in LN_BAD])
def test_bad_descriptor(kind, field, value, status):
    queries = dict(conv=("conv_bwd_workspace_bytes",), ssm=("ssm_saved_bytes", "ssm_workspace_bytes", "ssm_bwd_workspace_bytes"),
                   layernorm=("layernorm_bwd_workspace_bytes",))[kind]
    for fn in NAMES:
        if fn.startswith(kind):
            d = desc_of(fn)
            setattr(d, field, value)
            assert call(fn, d, fakes(fn)) == status, fn
    for q in queries:
        with pytest.raises(osr.OSRError):
            getattr(osr, "lattice_osr_" + q)(d)


@pytest.mark.parametrize("fn", NAMES)
def test_null_descriptor(fn):
    assert call(fn, None, fakes(fn)) == NULL


REQUIRED = dict(conv_fwd=("x", "w", "y"), conv_bwd=("x", "w", "dy", "dx", "ws"), conv_step=("x", "w", "hist_in", "hist_out", "y"),
                ssm_fwd=("x", "dt", "A", "Bm", "Cm", "y"),
                ssm_bwd=("x", "dt", "A", "Bm", "Cm", "saved", "dy", "dx", "ddt", "dB", "dC", "dz", "ws"),
                ssm_step=("x", "dt", "A", "Bm", "Cm", "state_in", "state_out", "y"), layernorm_fwd=("x", "z"),
                layernorm_bwd=("x", "dz", "ws"))


@pytest.mark.parametrize("fn", NAMES)
def test_null_pointers(fn):
    for n in REQUIRED[fn]:
        assert call(fn, desc_of(fn), {**fakes(fn), n: None}) == NULL, n


def test_operands_without_their_use():
    b = fakes("ssm_bwd")
    for n, g in (("z", "dz"), ("skip", "dskip"), ("dt_bias", "ddt_bias")):
        assert call("ssm_bwd", desc_of("ssm"), {**b, n: None}) == NO, g
    lf, lb = fakes("layernorm_fwd"), fakes("layernorm_bwd")
    assert call("layernorm_fwd", desc_of("layernorm"), {**lf, "y": None}) == NO          # x_out without y
    assert call("layernorm_bwd", desc_of("layernorm"), {**lb, "y": None}) == NO          # dy without y
    assert call("layernorm_bwd", desc_of("layernorm"), {**lb, "dx": None, "dy": None}) == NULL
    assert call("conv_step", desc_of("conv", T=2), fakes("conv_step")) == SHAPE
    assert call("conv_step", desc_of("conv", W=1), fakes("conv_step")) == SHAPE
    assert call("ssm_step", desc_of("ssm", T=2), fakes("ssm_step")) == SHAPE


@pytest.mark.parametrize("fn", NAMES)
def test_misaligned(fn):
    d = desc_of(fn)
    for n in names_of(fn, d):
        p = {**fakes(fn), "ws": WS}
        p[n] += 1
        assert call(fn, d, p) == osr.ERR_ALIGN, n


@pytest.mark.parametrize("fn", NAMES)
def test_aliases(fn):
    d = desc_of(fn)
    for out in OUTS[fn]:
        for other in names_of(fn, d):
            if other == out:
                continue
            p = {**fakes(fn), "ws": WS}
            p[out] = p[other] + (16 if (fn, out, other) in SAME or (fn, other, out) in SAME else 0)
            assert call(fn, d, p) == osr.ERR_ALIAS, (out, other)


def test_rows_apart_reach_to_their_last_element():
    """An input with a stride between its rows ends with its last row, not with that row's stride; an output
    inside that reach, between the rows too, is refused."""
    d = desc_of("ssm", T=3, D=64, z_row=200)
    p = fakes("ssm_fwd")
    reach = ((2 * 3 - 1) * 200 + 64) * 2  # bf16
    for at, ok in ((reach - 4, False), (70 * 2 * 4, False)):
        assert call("ssm_fwd", d, {**p, "y": p["z"] + at}) == osr.ERR_ALIAS
    # just behind: past this check, so that the next one (the workspace's overlap) answers
    assert call("ssm_fwd", d, {**p, "y": p["z"] + reach, "state_out": p["x"]}) == osr.ERR_ALIAS
    c = desc_of("conv", T=3, x_row=128)
    q = fakes("conv_fwd")
    assert call("conv_fwd", c, {**q, "y": q["x"] + ((2 * 3 - 1) * 128 + 64) * 2 - 2}) == osr.ERR_ALIAS


def test_sizes_of_saved_and_workspaces():
    for B, T, D, N in ((1, 1, 1, 1), (2, 16, 64, 16), (3, 17, 66, 5), (1, 65536, 2048, 16)):
        d = osr.make_ssm_desc(B, T, D, N)
        need = B * ((T + 15) // 16) * N * D * 4
        assert osr.lattice_osr_ssm_saved_bytes(d) == need
        if T == 1:
            continue
        assert call("ssm_fwd", d, fakes("ssm_fwd"), saved=need - 1) == osr.ERR_WORKSPACE
        assert call("ssm_bwd", d, fakes("ssm_bwd"), saved=need - 1) == osr.ERR_WORKSPACE
        assert call("ssm_bwd", d, fakes("ssm_bwd"), saved=1 << 50,
                    ws=osr.lattice_osr_ssm_bwd_workspace_bytes(d) - 1) == osr.ERR_WORKSPACE
    c = desc_of("conv", T=300)
    assert call("conv_bwd", c, fakes("conv_bwd"), ws=osr.lattice_osr_conv_bwd_workspace_bytes(c) - 1) == osr.ERR_WORKSPACE
    n = desc_of("layernorm")
    need = osr.lattice_osr_layernorm_bwd_workspace_bytes(n)
    assert need > 0 and call("layernorm_bwd", n, fakes("layernorm_bwd"), ws=need - 1) == osr.ERR_WORKSPACE


def test_size_limits():
    """The largest sizes inside each limit are taken, the next are refused."""
    ok = osr.lattice_osr_ssm_saved_bytes
    assert ok(osr.make_ssm_desc((1 << 22) - 1, 1, 64, 1)) > 0
    with pytest.raises(osr.OSRError):
        ok(osr.make_ssm_desc(1 << 22, 1, 64, 1))
    with pytest.raises(osr.OSRError):
        ok(osr.make_ssm_desc(1 << 21, 1, 65, 1))
    with pytest.raises(osr.OSRError):  # one group's 2 channels are a block of their own
        ok(osr.make_ssm_desc(4, 1, 1 << 21, 1, 1 << 20))
    assert ok(osr.make_ssm_desc(1, 1 << 30, 1, 1)) > 0
    assert osr.lattice_osr_conv_bwd_workspace_bytes(osr.make_conv_desc(1, 1 << 30, 31, 4)) > 0
    with pytest.raises(osr.OSRError):
        osr.lattice_osr_conv_bwd_workspace_bytes(osr.make_conv_desc(1, 1 << 30, 32, 4))


@pytest.mark.parametrize("B,T,D", [(1 << 26, 1, 16), (1 << 26, 128, 1), ((1 << 26) - 1, 129, 1), (1 << 19, 1 << 14, 3),
                                   ((1 << 31) - 1, 1, 1)])
def test_convolution_backward_runs(B, T, D):
    """B ceil(T / 128) runs of 64 threads each are a launch of fewer than 2^32, whatever D is: what has more of them is
    refused by the backward and its workspace query before anything is asked for, and taken by the forward."""
    assert B * -(-T // 128) >= 1 << 26 and B * -(-T // 16) * D < 1 << 31
    d = osr.make_conv_desc(B, T, D, 1)
    # buffers further apart than the largest of them
    far = lambda fn: {n: BASE + i * (1 << 44) for i, n in enumerate(NAMES[fn])}
    assert call("conv_bwd", d, far("conv_bwd"), ws=1 << 50) == SHAPE
    with pytest.raises(osr.OSRError):
        osr.lattice_osr_conv_bwd_workspace_bytes(d)
    p = far("conv_fwd")
    assert call("conv_fwd", d, {**p, "y": p["x"]}) == osr.ERR_ALIAS  # past the check of the sizes
    inside = osr.make_conv_desc((1 << 26) - 1, 1, 16, 1)
    assert osr.lattice_osr_conv_bwd_workspace_bytes(inside) == ((1 << 26) - 1) * 2 * 16 * 4


# -------------------------------------------------------------- binding --
B, T, D, N = 2, 6, 24, 5
BF = torch.bfloat16


def _raises(msg, fn, *a, **k):
    with pytest.raises(ValueError, match=msg):
        fn(*a, **k)


def _z(*s, dtype=BF):
    return torch.zeros(s, dtype=dtype)


def test_ssm_binding_checks():
    f32 = torch.float32
    a = dict(x=_z(B, T, D), dt=_z(B, T, D), A=_z(D, N, dtype=f32), B=_z(B, T, N), C=_z(B, T, N))
    f = osr.lattice_osr_ssm_fwd
    _raises("GPU", f, **a)
    _raises(r"\[B,T,D\] or \[B,T,H,d\]", f, **{**a, "x": _z(T, D)})
    _raises("float32 or bfloat16", f, **{**a, "x": _z(B, T, D).half()})
    _raises("dt has shape", f, **{**a, "dt": _z(B, T, D + 1)})
    _raises("dt is", f, **{**a, "dt": _z(B, T, D, dtype=f32)})
    _raises("A is .D,N.", f, **{**a, "A": _z(N, dtype=f32)})
    _raises("A has shape", f, **{**a, "A": _z(D + 1, N, dtype=f32)})
    _raises("A is torch", f, **{**a, "A": _z(D, N)})
    _raises("B and C are", f, **{**a, "B": _z(B, T)})
    _raises("B has shape", f, **{**a, "B": _z(B, T, N + 1)})
    _raises("C has shape", f, **{**a, "B": _z(B, T, 2, N)})
    _raises("C is", f, **{**a, "C": _z(B, T, N, dtype=f32)})
    _raises("D has shape", f, **a, D=_z(N, dtype=f32))
    _raises("dt_bias is", f, **a, dt_bias=_z(D))
    _raises("z has shape", f, **a, z=_z(B, T, D, 1))
    _raises("lengths is", f, **a, lengths=torch.zeros(B, dtype=torch.int64))
    _raises("segments has shape", f, **a, segments=torch.zeros(B, T + 1, dtype=torch.int32))
    _raises("segments is", f, **a, segments=torch.zeros(B, T))
    _raises("state_in has shape", f, **a, state_in=_z(B, N, D, dtype=f32))
    _raises("state_out is", f, **a, state_out=_z(B, D, N))
    _raises("y is", f, **a, y=_z(B, T, D))
    _raises("float32 or bfloat16", f, **a, y_dtype=torch.float16)
    wide = _z(B, T, 2 * D)
    _raises("GPU", f, **{**a, "x": wide[..., D:], "dt": wide[..., :D]})
    _raises("stride between tokens", f, **{**a, "x": _z(B, T, 2 * D)[..., ::2]})
    _raises("stride between tokens", f, **{**a, "x": _z(T, B, D).transpose(0, 1)})
    _raises("stride between tokens", f, **{**a, "x": _z(B, T, 1).expand(B, T, D)})
    _raises("stride between tokens", f, **{**a, "x": _z(B, 1, D).expand(B, T, D)})
    _raises("stride between tokens", f, **{**a, "dt": _z(B, 2 * T, D)[:, :T]})
    _raises("must be contiguous", f, **{**a, "A": _z(N, D, dtype=f32).t()})
    four = dict(x=_z(B, T, 3, 8), dt=_z(B, T, 3, 8), A=_z(3, 8, N, dtype=f32), B=_z(B, T, 3, N), C=_z(B, T, 3, N))
    _raises("GPU", f, **four, state_in=_z(B, 3, 8, N, dtype=f32))
    _raises("state_in has shape", f, **four, state_in=_z(B, D, N, dtype=f32))
    g = osr.lattice_osr_ssm_bwd
    saved = torch.zeros(1000, dtype=torch.uint8)
    _raises("saved", g, **a, dy=_z(B, T, D), saved=None)
    _raises("dy has shape", g, **a, dy=_z(B, T, N), saved=saved)
    _raises("dstate_out has shape", g, **a, dy=_z(B, T, D), dstate_out=_z(B), saved=saved)
    _raises("grads lacks ddt", g, **a, dy=_z(B, T, D), saved=saved, grads={"dx": _z(B, T, D, dtype=f32)})
    _raises("dx is", g, **a, dy=_z(B, T, D), saved=saved, grads={"dx": _z(B, T, D)})
    _raises("GPU", g, **a, dy=_z(B, T, D), saved=saved)
    s = osr.lattice_osr_ssm_step
    _raises("state_in has shape", s, **a, state_in=_z(B, D, dtype=f32))
    _raises("state_in: the state", s, **a, state_in=None)
    _raises("GPU", s, **a, state_in=_z(B, D, N, dtype=f32))


def test_conv_binding_checks():
    f32 = torch.float32
    x, w = _z(B, T, D), _z(D, 4, dtype=f32)
    f = osr.lattice_osr_conv_fwd
    _raises("GPU", f, x, w)
    _raises("w is .D,W.", f, x, w[0])
    _raises("w has shape", f, x, _z(D + 1, 4, dtype=f32))
    _raises("w is torch", f, x, _z(D, 4))
    _raises("bias has shape", f, x, w, _z(4, dtype=f32))
    _raises("hist_in has shape", f, x, w, None, _z(B, 4, D))
    _raises("hist_in is", f, x, w, None, _z(B, 3, D, dtype=f32))
    _raises("hist_out has shape", f, x, w, hist_out=_z(B, 3, D + 1))
    _raises("y is", f, x, w, y=_z(B, T, D, dtype=f32))
    _raises("stride between tokens", f, _z(B, D, T).transpose(1, 2), w)
    _raises("lengths has shape", f, x, w, lengths=torch.zeros(B + 1, dtype=torch.int32))
    g = osr.lattice_osr_conv_bwd
    _raises("dy has shape", g, x, w, _z(B, T, D + 1))
    _raises("dhist_out is", g, x, w, x, None, None, _z(B, 3, D))
    _raises("grads lacks dw", g, x, w, x, grads={"dx": _z(B, T, D, dtype=f32)})
    _raises("GPU", g, x, w, x)
    s = osr.lattice_osr_conv_step
    _raises("hist_in: the history", s, x[:, :1].contiguous(), w, None)
    _raises("GPU", s, x[:, :1].contiguous(), w, _z(B, 3, D))


def test_layernorm_binding_checks():
    x, y = torch.zeros(5, D), _z(5, D)
    w = torch.zeros(D)
    f, g = osr.lattice_osr_layernorm_fwd, osr.lattice_osr_layernorm_bwd
    _raises("GPU", f, x, y, w=w)
    _raises("y has shape", f, x, y[:4])
    _raises("w has shape", f, x, y, w=torch.zeros(D + 1))
    _raises("b is", f, x, y, b=w.double())
    _raises("z_dtype", f, x, y, z_dtype=torch.float32)
    _raises("z is", f, x, y, z=x)
    _raises("x_out is", f, x, y, x_out=y)
    _raises("must be contiguous", f, torch.zeros(D, 5).t())
    _raises("float32 or bfloat16", f, x.double())
    _raises("float32 or bfloat16", f, x, z_dtype=torch.float16)
    _raises("dz: the gradient", g, x, y)
    _raises("dz is", g, x, y, None, x)
    _raises("dx_out has shape", g, x, y, x[:4], y)
    _raises("grads lacks dy", g, x, y, x, y, grads={"dx": x})
    _raises("GPU", g, x, y, x, y, w=w)
