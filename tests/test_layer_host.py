"""Host-only checks of the layer operators (lattice_osr_scan_*, lattice_osr_norm_*):
argument checks of the C ABI with the documented status codes, before any HIP
call, and of the Python binding (no GPU needed)."""
import ctypes
import math

import pytest
import torch

from compressed_memory_linear_amd import osr

# Fake device addresses: only compared and range-checked on the host, because
# every case below fails validation first.
BASE, GAP = 1 << 40, 1 << 34


def _lib():
    return osr.load_library()


def _fake(*names):
    return {n: BASE + i * GAP for i, n in enumerate(names)}


# ----------------------------------------------------------------- scan --
FWD = ("v", "mu_logit", "gamma_logit", "lengths", "state_in", "state_out", "y", "saved")
BWD = ("v", "mu_logit", "gamma_logit", "lengths", "saved", "dy", "dstate_out", "dv", "dmu_logit", "dgamma_logit",
       "dstate_in")
STEP = ("v", "mu_logit", "gamma_logit", "state_in", "state_out", "y")
WS = BASE + 40 * GAP


def _fwd(d, p, saved_bytes=None, ws=WS, ws_bytes=1 << 33):
    if saved_bytes is None:
        saved_bytes = 1 << 33
    return _lib().lattice_osr_scan_fwd(ctypes.byref(d), *[p[n] for n in FWD], saved_bytes, ws, ws_bytes, None)


def _bwd(d, p, saved_bytes=1 << 33, ws=WS, ws_bytes=1 << 33):
    return _lib().lattice_osr_scan_bwd(ctypes.byref(d), *[p[n] for n in BWD[:5]], saved_bytes, *[p[n] for n in BWD[5:]],
                                       ws, ws_bytes, None)


def _step(d, p):
    return _lib().lattice_osr_scan_step(ctypes.byref(d), *[p[n] for n in STEP], None)


@pytest.mark.parametrize("field,value,status", [
    ("B", 0, osr.ERR_SHAPE), ("T", 0, osr.ERR_SHAPE), ("D", 0, osr.ERR_SHAPE), ("B", -1, osr.ERR_SHAPE),
    ("T", -3, osr.ERR_SHAPE), ("D", (1 << 20) + 1, osr.ERR_SHAPE), ("T", (1 << 30) + 1, osr.ERR_SHAPE),
    ("B", 1 << 22, osr.ERR_SHAPE),
    ("in_dtype", 2, osr.ERR_UNSUPPORTED), ("y_dtype", -1, osr.ERR_UNSUPPORTED), ("grad_dtype", 5, osr.ERR_UNSUPPORTED),
    ("input_weight", 3, osr.ERR_UNSUPPORTED), ("input_weight", -1, osr.ERR_UNSUPPORTED),
])
def test_scan_bad_descriptor(field, value, status):
    d = osr.make_scan_desc(2, 1, 64)
    setattr(d, field, value)
    assert _fwd(d, _fake(*FWD)) == status
    assert _bwd(d, _fake(*BWD)) == status
    assert _step(d, _fake(*STEP)) == status
    for f in (osr.lattice_osr_scan_saved_bytes, osr.lattice_osr_scan_workspace_bytes):
        with pytest.raises(osr.OSRError):
            f(d)


def test_scan_null_pointers():
    d = osr.make_scan_desc(2, 1, 64)
    assert _lib().lattice_osr_scan_fwd(None, *[BASE] * 8, 0, None, 0, None) == osr.ERR_NULL
    for n in ("v", "mu_logit", "y"):
        assert _fwd(d, {**_fake(*FWD), n: None}) == osr.ERR_NULL
    for n in ("v", "mu_logit", "saved", "dy", "dv", "dmu_logit", "dgamma_logit"):
        assert _bwd(d, {**_fake(*BWD), n: None}) == osr.ERR_NULL
    assert _bwd(d, {**_fake(*BWD), "gamma_logit": None}) == osr.ERR_UNSUPPORTED
    for n in ("v", "mu_logit", "state_in", "state_out", "y"):
        assert _step(d, {**_fake(*STEP), n: None}) == osr.ERR_NULL
    assert _lib().lattice_osr_scan_saved_bytes(None) == ctypes.c_size_t(-1).value


def test_scan_step_takes_one_token():
    assert _step(osr.make_scan_desc(2, 2, 64), _fake(*STEP)) == osr.ERR_SHAPE


def test_scan_saved_size_and_bounds():
    """One state per 128 tokens, begun ones included."""
    for B, T, D in ((1, 1, 1), (2, 128, 64), (3, 129, 65), (1, 65536, 2048)):
        d = osr.make_scan_desc(B, T, D)
        need = B * ((T + 127) // 128) * D * 4
        assert osr.lattice_osr_scan_saved_bytes(d) == need
        assert _fwd(d, _fake(*FWD), saved_bytes=need - 1) == osr.ERR_WORKSPACE
        assert _bwd(d, _fake(*BWD), saved_bytes=need - 1) == osr.ERR_WORKSPACE


def test_scan_misaligned():
    d = osr.make_scan_desc(2, 1, 64, osr.BF16, osr.F32, osr.F32)
    for names, call in ((FWD, _fwd), (BWD, _bwd), (STEP, _step)):
        for n in names:
            p = _fake(*names)
            p[n] += 1
            assert call(d, p) == osr.ERR_ALIGN, n
            if n not in ("v", "mu_logit", "gamma_logit"):  # bf16 here: 2-byte elements
                p[n] += 1
                assert call(d, p) == osr.ERR_ALIGN, n


def test_scan_aliases():
    d = osr.make_scan_desc(2, 1, 64)
    n = 2 * 64
    for out in ("y", "state_out", "saved"):
        for other in FWD:
            if other == out:
                continue
            p = _fake(*FWD)
            p[out] = p[other]
            if {out, other} == {"state_out", "state_in"}:
                p[out] += 8  # a partial overlap: only the very state may be updated in place
            assert _fwd(d, p) == osr.ERR_ALIAS, (out, other)
    for out in BWD[7:]:
        for other in BWD:
            if other != out:
                p = _fake(*BWD)
                p[out] = p[other]
                assert _bwd(d, p) == osr.ERR_ALIAS, (out, other)
    p = _fake(*STEP)
    p["y"] = p["state_out"] + n * 4 - 4
    assert _step(d, p) == osr.ERR_ALIAS
    p = _fake(*STEP)
    p["state_out"] = p["state_in"] + 4
    assert _step(d, p) == osr.ERR_ALIAS


# ---------------------------------------------------------------- norms --
NF = ("y", "gate", "x", "w_post", "scale", "w_pre", "x_out", "z")
NB = ("y", "gate", "x", "w_post", "scale", "w_pre", "dx_out", "dz", "dy", "dgate", "dx", "dw_post", "dscale", "dw_pre")


def _nf(d, p):
    return _lib().lattice_osr_norm_fwd(ctypes.byref(d), *[p[n] for n in NF], None)


def _nb(d, p, ws=WS, ws_bytes=1 << 33):
    return _lib().lattice_osr_norm_bwd(ctypes.byref(d), *[p[n] for n in NB], ws, ws_bytes, None)


def _nd(**kw):
    return osr.make_norm_desc(4, 64, **{"gate_kind": osr.GATE_GELU, **kw})


@pytest.mark.parametrize("field,value,status", [
    ("R", 0, osr.ERR_SHAPE), ("D", 0, osr.ERR_SHAPE), ("R", -1, osr.ERR_SHAPE), ("D", 16385, osr.ERR_UNSUPPORTED),
    ("in_dtype", 2, osr.ERR_UNSUPPORTED), ("res_dtype", 2, osr.ERR_UNSUPPORTED), ("grad_dtype", 2, osr.ERR_UNSUPPORTED),
    ("gate_kind", 3, osr.ERR_UNSUPPORTED), ("gate_kind", -1, osr.ERR_UNSUPPORTED),
    ("post_norm", 2, osr.ERR_UNSUPPORTED), ("pre_norm", -1, osr.ERR_UNSUPPORTED),
    ("eps", 0.0, osr.ERR_UNSUPPORTED), ("eps", -1e-6, osr.ERR_UNSUPPORTED), ("eps", math.nan, osr.ERR_UNSUPPORTED),
    ("eps", math.inf, osr.ERR_UNSUPPORTED), ("eps", 1e-39, osr.ERR_UNSUPPORTED),
])
def test_norm_bad_descriptor(field, value, status):
    d = _nd()
    setattr(d, field, value)
    assert _nf(d, _fake(*NF)) == status
    assert _nb(d, _fake(*NB)) == status
    with pytest.raises(osr.OSRError):
        osr.lattice_osr_norm_bwd_workspace_bytes(d)


def test_norm_operands():
    NULL, NO = osr.ERR_NULL, osr.ERR_UNSUPPORTED
    f, b = _fake(*NF), _fake(*NB)
    assert _nf(_nd(), {**f, "y": None, "x": None}) == NULL
    assert _nf(_nd(), {**f, "gate": None}) == NULL                                   # a gate kind without a gate
    assert _nf(_nd(gate_kind=osr.GATE_NONE), f) == NO                                # a gate without its kind
    assert _nf(_nd(post_norm=0), f) == NO                                            # w_post without its norm
    assert _nf(_nd(pre_norm=0), {**f, "z": None}) == NO                              # w_pre without its norm
    assert _nf(_nd(), {**f, "z": None}) == NULL
    assert _nf(_nd(pre_norm=0), {**f, "w_pre": None}) == NO                          # z without its norm
    assert _nf(_nd(pre_norm=0), {**f, "w_pre": None, "z": None, "x_out": None}) == NULL
    only_x = {**f, "y": None, "gate": None, "w_post": None, "scale": None}
    assert _nf(_nd(gate_kind=0, post_norm=0), only_x) == NO                          # x_out without y
    assert _nf(_nd(gate_kind=0), {**only_x, "x_out": None}) == NO                    # post_norm without y
    assert _nf(_nd(gate_kind=0, post_norm=0), {**only_x, "x_out": None, "scale": f["scale"]}) == NO
    assert _nf(_nd(gate_kind=0, post_norm=0, pre_norm=0), {**only_x, "x_out": None, "z": None, "w_pre": None}) == NO
    for n in ("dy", "dgate", "dz"):
        assert _nb(_nd(), {**b, n: None}) == NULL, n
    assert _nb(_nd(pre_norm=0), {**b, "w_pre": None, "dz": None, "dw_pre": None, "dx_out": None}) == NULL
    assert _nb(_nd(pre_norm=0), {**b, "w_pre": None, "dw_pre": None}) == NO          # dz without its norm
    assert _nb(_nd(post_norm=0), {**b, "w_post": None}) == NO                        # dw_post without its norm
    assert _nb(_nd(), {**b, "x": None}) == NO                                        # dx without x
    assert _nb(_nd(), b, ws=None) == NULL
    need = osr.lattice_osr_norm_bwd_workspace_bytes(_nd())
    assert need > 0 and _nb(_nd(), b, ws_bytes=need - 1) == osr.ERR_WORKSPACE
    assert _nb(_nd(), b, ws=WS + 2) == osr.ERR_ALIGN


def test_norm_misaligned_and_aliases():
    d = _nd()
    for names, call, outs, same in ((NF, _nf, ("x_out", "z"), ("x_out", "x")),
                                    (NB, _nb, ("dy", "dgate", "dx", "dw_post", "dscale", "dw_pre"), ("dx", "dx_out"))):
        for n in names:
            p = _fake(*names)
            p[n] += 1
            assert call(d, p) == osr.ERR_ALIGN, n
        for out in outs:
            for other in names:
                if other == out:
                    continue
                p = _fake(*names)
                p[out] = p[other] + (16 if (out, other) == same else 0)
                assert call(d, p) == osr.ERR_ALIAS, (out, other)
    p = _fake(*NB)
    assert _nb(d, p, ws=p["dy"]) == osr.ERR_ALIAS


# -------------------------------------------------------------- binding --
B, T, D = 2, 6, 24


def _x(dtype=torch.bfloat16):
    return dict(v=torch.zeros(B, T, D, dtype=dtype), mu_logit=torch.zeros(B, T, D, dtype=dtype))


def _raises(msg, fn, *a, **k):
    with pytest.raises(ValueError, match=msg):
        fn(*a, **k)


def test_scan_binding_checks():
    x = _x()
    st = torch.zeros(B, D)
    f = osr.lattice_osr_scan_fwd
    _raises("GPU", f, **x)
    _raises("mu_logit has shape", f, x["v"], torch.zeros(B, T, D + 1, dtype=torch.bfloat16))
    _raises("mu_logit is", f, x["v"], torch.zeros(B, T, D))
    _raises("gamma_logit has shape", f, **x, gamma_logit=torch.zeros(B, T, dtype=torch.bfloat16))
    _raises("must be contiguous", f, torch.zeros(B, T, 2 * D, dtype=torch.bfloat16)[..., :D], x["mu_logit"])
    _raises("state_in has shape", f, **x, state_in=torch.zeros(B, D + 1))
    _raises("state_in is", f, **x, state_in=torch.zeros(B, D, dtype=torch.bfloat16))
    _raises("state_out has shape", f, **x, state_out=torch.zeros(B + 1, D))
    _raises("lengths is", f, **x, lengths=torch.zeros(B, dtype=torch.int64))
    _raises("lengths has shape", f, **x, lengths=torch.zeros(B + 1, dtype=torch.int32))
    _raises("y is", f, **x, y=torch.zeros(B, T, D, dtype=torch.bfloat16))
    _raises("y_dtype", f, **x, y_dtype=torch.float16)
    _raises("float32 or bfloat16", f, x["v"].half(), x["mu_logit"].half())
    _raises(r"\[B,T,D\] or \[B,T,H,d\]", f, x["v"][0], x["mu_logit"][0])
    four = torch.zeros(B, T, 3, 8, dtype=torch.bfloat16)
    _raises("state_in has shape", f, four, four, state_in=st)
    _raises("GPU", f, four, four, state_in=torch.zeros(B, 3, 8))
    g = osr.lattice_osr_scan_bwd
    saved, dy = torch.zeros(1000, dtype=torch.uint8), torch.zeros(B, T, D)
    _raises("saved", g, **x, dy=dy, saved=None)
    _raises("dy has shape", g, **x, dy=torch.zeros(B, T, D + 1), saved=saved)
    _raises("dstate_out has shape", g, **x, dy=dy, dstate_out=torch.zeros(B), saved=saved)
    _raises("grads lacks dmu_logit", g, **x, dy=dy, saved=saved, grads={"dv": torch.zeros(B, T, D)})
    _raises("dv is", g, **x, dy=dy, saved=saved, grads={"dv": torch.zeros(B, T, D)}, grad_dtype=torch.bfloat16)
    _raises("GPU", g, **x, dy=dy, saved=saved)
    s = osr.lattice_osr_scan_step
    _raises("state_in has shape", s, **x, state_in=torch.zeros(D))
    _raises("GPU", s, **x, state_in=st)


def test_norm_binding_checks():
    y, x = torch.zeros(5, D, dtype=torch.bfloat16), torch.zeros(5, D)
    w = torch.zeros(D)
    f, g = osr.lattice_osr_norm_fwd, osr.lattice_osr_norm_bwd
    _raises("pass y, x or both", f)
    _raises("x has shape", f, y, torch.zeros(4, D))
    _raises("gate is", f, y, x, gate=torch.zeros(5, D))
    _raises("GATE_NONE", f, y, x, gate=y, gate_kind=osr.GATE_NONE)
    _raises("w_post has shape", f, y, x, w_post=torch.zeros(D + 1))
    _raises("w_pre is", f, y, x, w_pre=w.double())
    _raises("must be contiguous", f, torch.zeros(D, 5, dtype=torch.bfloat16).t(), x)
    _raises("x_out is", f, y, x, x_out=torch.zeros(5, D, dtype=torch.bfloat16))
    _raises("z is", f, y, x, z=torch.zeros(5, D))
    _raises("z_dtype", f, y, x, z_dtype=torch.float32)
    _raises("x_dtype", f, y, x, x_dtype=torch.bfloat16)
    _raises("float32 or bfloat16", f, y.half(), x)
    _raises("GPU", f, y, x, w_post=w)
    _raises("dx_out is", g, y, x, y, y)
    _raises("dz has shape", g, y, x, x, torch.zeros(5, D + 1, dtype=torch.bfloat16))
    _raises("grads lacks dx", g, y, x, x, y, grads={"dy": torch.zeros(5, D)})
    _raises("GPU", g, y, x, x, y, w_post=w, w_pre=w)


def test_scan_workspace():
    """None for a single tile; required, sized, 16-byte aligned and apart from every argument otherwise."""
    assert osr.lattice_osr_scan_workspace_bytes(osr.make_scan_desc(3, 128, 100)) == 0
    d = osr.make_scan_desc(3, 200, 100)
    need = osr.lattice_osr_scan_workspace_bytes(d)
    assert need > 0
    for names, call in ((FWD, _fwd), (BWD, _bwd)):
        p = _fake(*names)
        assert call(d, p, ws=None) == osr.ERR_NULL
        assert call(d, p, ws_bytes=need - 1) == osr.ERR_WORKSPACE
        assert call(d, p, ws=WS + 8) == osr.ERR_ALIGN
        for n in names:
            assert call(d, p, ws=p[n]) == osr.ERR_ALIAS, n


@pytest.mark.parametrize("B,D,tiles", [(1, 64, (1 << 22) - 1), (1, 1, (1 << 21) + 1), (3, 64, 1398101), (1, 129, 1398101),
                                       ((1 << 22) - 1, 64, 1), (5, 100, 419430)])
def test_scan_size_limit(B, D, tiles):
    """B ceil(D / 64) ceil(T / 128) below 2^22, that product itself: the largest T inside is taken, one token more
    is refused where it begins the tile that reaches the limit."""
    chains = B * ((D + 63) // 64)
    assert chains * tiles < 1 << 22
    T = tiles * 128
    assert osr.lattice_osr_scan_saved_bytes(osr.make_scan_desc(B, T, D)) == B * tiles * D * 4
    if chains * (tiles + 1) >= 1 << 22:
        d = osr.make_scan_desc(B, T + 1, D)
        with pytest.raises(osr.OSRError):
            osr.lattice_osr_scan_saved_bytes(d)
        assert _fwd(d, _fake(*FWD)) == osr.ERR_SHAPE
