"""Python binding of liblattice_osr.so (include/lattice_osr.h).

Argument marshalling only: every step of the recurrence runs in the library's
HIP kernels.  Tensors are PyTorch device tensors (PyTorch provides device
memory and the stream); the functions keep the C entry points' names.

If the library has not been built (``python -m compressed_memory_linear_amd.build``)
the first call raises; there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblattice_osr.so")

F32, BF16 = 0, 1
MODE_DEC, MODE_SIM, MODE_ENC = 0, 1, 2
LIN2, LIN1 = 0, 1
SCHED_AUTO, SCHED_SPLIT, SCHED_FUSED = 0, 1, 2
PAIRS_AUTO, PAIRS_OFF = 0, 1
WGS_AUTO, WGS_ONE = 0, 1
OVERLAP_AUTO, OVERLAP_OFF = 0, 1
BWD_AUTO, BWD_WALK, BWD_CHUNK = 0, 1, 2
SCAN_ONE, SCAN_COMPLEMENT, SCAN_NORM = 0, 1, 2
GATE_NONE, GATE_GELU, GATE_SILU = 0, 1, 2
CONV_NONE, CONV_SILU = 0, 1

OK = 0
ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_LAUNCH, ERR_ALIAS, ERR_ALIGN = -1, -2, -3, -4, -5, -6, -7

EXPORTED = ("lattice_osr_fwd_chunked", "lattice_osr_fwd_recurrent", "lattice_osr_decode_step",
            "lattice_osr_workspace_bytes", "lattice_osr_status_string", "lattice_osr_abi_version",
            "lattice_osr_bwd_chunked", "lattice_osr_bwd_workspace_bytes", "lattice_osr_glue_pre",
            "lattice_osr_glue_post", "lattice_osr_fwd_chunked_gated", "lattice_osr_fwd_chunked_noalloc",
            "lattice_osr_fwd_chunked_save", "lattice_osr_bwd_chunked_saved", "lattice_osr_scan_fwd",
            "lattice_osr_scan_bwd", "lattice_osr_scan_step", "lattice_osr_scan_saved_bytes",
            "lattice_osr_scan_workspace_bytes", "lattice_osr_norm_fwd", "lattice_osr_norm_bwd",
            "lattice_osr_norm_bwd_workspace_bytes", "lattice_osr_conv_fwd", "lattice_osr_conv_bwd",
            "lattice_osr_conv_step", "lattice_osr_conv_bwd_workspace_bytes", "lattice_osr_ssm_fwd",
            "lattice_osr_ssm_bwd", "lattice_osr_ssm_step", "lattice_osr_ssm_saved_bytes",
            "lattice_osr_ssm_workspace_bytes", "lattice_osr_ssm_bwd_workspace_bytes", "lattice_osr_layernorm_fwd",
            "lattice_osr_layernorm_bwd", "lattice_osr_layernorm_bwd_workspace_bytes")
NOALLOC_SCRATCH_BYTES = 64 << 20


class lattice_osr_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "T", "H", "m", "d", "gamma_per_slot", "in_dtype", "y_dtype", "mode", "linearisation",
                 "schedule", "chain_pairs", "chain_wgs", "readout_overlap", "bwd_form")]


class lattice_osr_scan_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "D", "in_dtype", "y_dtype", "grad_dtype", "input_weight")]


class lattice_osr_norm_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("R", "D", "in_dtype", "res_dtype", "grad_dtype", "gate_kind", "post_norm", "pre_norm")] + \
               [("eps", ctypes.c_float)]


class lattice_osr_conv_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "D", "W", "act", "in_dtype", "y_dtype", "grad_dtype", "x_row")]


class lattice_osr_ssm_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "D", "N", "G", "in_dtype", "y_dtype", "grad_dtype", "softplus",
                                             "x_row", "dt_row", "z_row", "b_row", "c_row")]


class lattice_osr_layernorm_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("R", "D", "in_dtype", "res_dtype", "grad_dtype")] + \
               [("eps", ctypes.c_float)]


class OSRError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: status {status} ({status_string(status)})")
        self.status = status


_lib = None


def load_library():
    """Load liblattice_osr.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m compressed_memory_linear_amd.build`")
        lib = ctypes.CDLL(LIB_PATH)
        vp, dp = ctypes.c_void_p, ctypes.POINTER(lattice_osr_desc)
        fwd = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        lib.lattice_osr_fwd_chunked.argtypes = [dp, ctypes.c_int32] + fwd[1:]
        lib.lattice_osr_fwd_chunked_gated.argtypes = [dp, ctypes.c_int32] + [vp] * 6 + fwd[6:]
        lib.lattice_osr_fwd_chunked_gated.restype = ctypes.c_int
        lib.lattice_osr_fwd_chunked_noalloc.argtypes = [dp, ctypes.c_int32] + [vp] * 9
        lib.lattice_osr_fwd_chunked_noalloc.restype = ctypes.c_int
        lib.lattice_osr_fwd_recurrent.argtypes = fwd
        lib.lattice_osr_decode_step.argtypes = fwd
        for f in ("lattice_osr_fwd_chunked", "lattice_osr_fwd_recurrent", "lattice_osr_decode_step"):
            getattr(lib, f).restype = ctypes.c_int
        lib.lattice_osr_bwd_chunked.argtypes = [dp, ctypes.c_int32] + [vp] * 15 + [ctypes.c_size_t, vp]
        lib.lattice_osr_bwd_chunked.restype = ctypes.c_int
        lib.lattice_osr_bwd_chunked_saved.argtypes = [dp, ctypes.c_int32] + [vp] * 15 + [ctypes.c_size_t, vp]
        lib.lattice_osr_bwd_chunked_saved.restype = ctypes.c_int
        lib.lattice_osr_fwd_chunked_save.argtypes = [dp, ctypes.c_int32] + fwd[1:]
        lib.lattice_osr_fwd_chunked_save.restype = ctypes.c_int
        lib.lattice_osr_bwd_workspace_bytes.argtypes = [dp, ctypes.c_int32]
        lib.lattice_osr_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.lattice_osr_workspace_bytes.argtypes = [dp, ctypes.c_int32]
        lib.lattice_osr_workspace_bytes.restype = ctypes.c_size_t
        lib.lattice_osr_glue_pre.argtypes = [dp] + [vp] * 15
        lib.lattice_osr_glue_pre.restype = ctypes.c_int
        lib.lattice_osr_glue_post.argtypes = [dp, vp, vp, vp, vp]
        lib.lattice_osr_glue_post.restype = ctypes.c_int
        sp, np_, sz = ctypes.POINTER(lattice_osr_scan_desc), ctypes.POINTER(lattice_osr_norm_desc), ctypes.c_size_t
        lib.lattice_osr_scan_fwd.argtypes = [sp] + [vp] * 8 + [sz, vp, sz, vp]
        lib.lattice_osr_scan_bwd.argtypes = [sp] + [vp] * 5 + [sz] + [vp] * 7 + [sz, vp]
        lib.lattice_osr_scan_step.argtypes = [sp] + [vp] * 7
        lib.lattice_osr_norm_fwd.argtypes = [np_] + [vp] * 9
        lib.lattice_osr_norm_bwd.argtypes = [np_] + [vp] * 15 + [sz, vp]
        for f in ("scan_fwd", "scan_bwd", "scan_step", "norm_fwd", "norm_bwd"):
            getattr(lib, "lattice_osr_" + f).restype = ctypes.c_int
        cp, mp, lp = (ctypes.POINTER(d) for d in (lattice_osr_conv_desc, lattice_osr_ssm_desc,
                                                  lattice_osr_layernorm_desc))
        lib.lattice_osr_conv_fwd.argtypes = [cp] + [vp] * 9
        lib.lattice_osr_conv_bwd.argtypes = [cp] + [vp] * 13 + [sz, vp]
        lib.lattice_osr_conv_step.argtypes = [cp] + [vp] * 7
        lib.lattice_osr_ssm_fwd.argtypes = [mp] + [vp] * 14 + [sz, vp, sz, vp]
        lib.lattice_osr_ssm_bwd.argtypes = [mp] + [vp] * 11 + [sz] + [vp] * 12 + [sz, vp]
        lib.lattice_osr_ssm_step.argtypes = [mp] + [vp] * 12
        lib.lattice_osr_layernorm_fwd.argtypes = [lp] + [vp] * 7
        lib.lattice_osr_layernorm_bwd.argtypes = [lp] + [vp] * 10 + [sz, vp]
        for f in ("conv_fwd", "conv_bwd", "conv_step", "ssm_fwd", "ssm_bwd", "ssm_step", "layernorm_fwd",
                  "layernorm_bwd"):
            getattr(lib, "lattice_osr_" + f).restype = ctypes.c_int
        for f, d in (("conv_bwd_workspace_bytes", cp), ("ssm_saved_bytes", mp), ("ssm_workspace_bytes", mp),
                     ("ssm_bwd_workspace_bytes", mp), ("layernorm_bwd_workspace_bytes", lp),
                     ("scan_saved_bytes", sp), ("scan_workspace_bytes", sp), ("norm_bwd_workspace_bytes", np_)):
            getattr(lib, "lattice_osr_" + f).argtypes = [d]
            getattr(lib, "lattice_osr_" + f).restype = sz
        lib.lattice_osr_status_string.argtypes = [ctypes.c_int]
        lib.lattice_osr_status_string.restype = ctypes.c_char_p
        lib.lattice_osr_abi_version.argtypes = []
        lib.lattice_osr_abi_version.restype = ctypes.c_int
        _lib = lib
    return _lib


def lattice_osr_abi_version() -> int:
    return int(load_library().lattice_osr_abi_version())


def status_string(status: int) -> str:
    return load_library().lattice_osr_status_string(int(status)).decode()


lattice_osr_status_string = status_string


def make_desc(B, T, H, m, d, gamma_per_slot=1, in_dtype=BF16, y_dtype=F32, mode=MODE_DEC, linearisation=LIN2,
              schedule=SCHED_AUTO, chain_pairs=PAIRS_AUTO, chain_wgs=WGS_AUTO, readout_overlap=OVERLAP_AUTO,
              bwd_form=BWD_AUTO):
    return lattice_osr_desc(B, T, H, m, d, gamma_per_slot, in_dtype, y_dtype, mode, linearisation, schedule,
                            chain_pairs, chain_wgs, readout_overlap, bwd_form)


def lattice_osr_workspace_bytes(desc: lattice_osr_desc, chunk_size: int) -> int:
    n = int(load_library().lattice_osr_workspace_bytes(ctypes.byref(desc), int(chunk_size)))
    if n == ctypes.c_size_t(-1).value:
        raise OSRError(ERR_SHAPE, "lattice_osr_workspace_bytes")
    return n


# ------------------------------------------------------------ marshalling --
_DT = {torch.float32: F32, torch.bfloat16: BF16}


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _shape_error(name, t, want):
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(want)}")


def _check_tensor(name, t, shape, dtype, device=None):
    """Shape, dtype and layout of one argument, then its device: the kernels
    index every buffer by the descriptor's sizes, so a mismatch would read or
    write past it on the GPU."""
    if (t.shape == shape and (dtype is None or t.dtype is dtype) and t.is_contiguous()
            and (device is None or t.device == device)):
        return
    if tuple(t.shape) != tuple(shape):
        _shape_error(name, t, shape)
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _check_cuda(*tensors):
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError("every tensor argument must be a GPU (cuda) tensor")


def _desc_from(q, k, v, gamma, mu, state_in, y_dtype, mode, linearisation=0, schedule=SCHED_AUTO,
               chain_pairs=PAIRS_AUTO, chain_wgs=WGS_AUTO, readout_overlap=OVERLAP_AUTO,
               bwd_form=BWD_AUTO) -> lattice_osr_desc:
    """Descriptor of a forward call, after checking every input against it:
    q, k [B,T,H,m]; v [B,T,H,d]; gamma [B,T,H,m] or [B,T,H]; mu [B,T,H]
    (all one dtype, float32 or bfloat16); state_in [B,H,m,d] float32; all
    contiguous, on one GPU."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q/k/gamma are [B,T,H,m], v is [B,T,H,d]")
    B, T, H, m = q.shape
    d = v.shape[-1]
    if q.dtype not in _DT:
        raise ValueError("inputs must be float32 or bfloat16")
    if y_dtype not in _DT:
        raise ValueError("y_dtype must be torch.float32 or torch.bfloat16")
    per_slot = 1 if gamma.dim() == 4 else 0
    _check_tensor("q", q, (B, T, H, m), q.dtype)
    _check_tensor("k", k, (B, T, H, m), q.dtype, q.device)
    _check_tensor("v", v, (B, T, H, d), q.dtype, q.device)
    _check_tensor("gamma", gamma, (B, T, H, m) if per_slot else (B, T, H), q.dtype, q.device)
    _check_tensor("mu", mu, (B, T, H), q.dtype, q.device)
    _check_tensor("state_in", state_in, (B, H, m, d), torch.float32, q.device)
    return make_desc(B, T, H, m, d, per_slot, _DT[q.dtype], _DT[y_dtype], mode, linearisation, schedule,
                     chain_pairs, chain_wgs, readout_overlap, bwd_form)


def _check_outputs(desc, q, state_in, state_out, y, y_dtype):
    """Caller-supplied outputs against the descriptor, then the device of
    every tensor."""
    if y is not None:
        _check_tensor("y", y, (desc.B, desc.T, desc.H, desc.d), y_dtype, q.device)
    if state_out is not None:
        _check_tensor("state_out", state_out, tuple(state_in.shape), torch.float32, q.device)
    _check_cuda(q)


def _outputs(desc, q, state_in, state_out, y, y_dtype):
    """Missing outputs are allocated (on the current stream, which the caller
    has set to the launch stream)."""
    if y is None:
        y = torch.empty((desc.B, desc.T, desc.H, desc.d), dtype=y_dtype, device=q.device)
    if state_out is None:
        state_out = torch.empty_like(state_in)
    return state_out, y


def _workspace(workspace, need, device):
    """The caller's workspace (a uint8 tensor on the inputs' device) or a new
    one of `need` bytes; returns (tensor or None, its size in bytes)."""
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous() or workspace.device != device:
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace, workspace.numel() * workspace.element_size()


def _launch_stream(stream):
    """The stream to launch on.  Temporaries (outputs, workspace) are
    allocated under it: the caching allocator then reuses their memory only
    in that stream's order, after the kernels that use it."""
    return torch.cuda.current_stream() if stream is None else stream


def lattice_osr_fwd_chunked(q, k, v, gamma, mu, state_in, chunk_size: int, *, mode: int = MODE_DEC,
                            y_dtype=torch.float32, state_out=None, y=None, workspace=None,
                            stream=None, linearisation: int = 0, schedule: int = SCHED_AUTO,
                            chain_pairs: int = PAIRS_AUTO, chain_wgs: int = WGS_AUTO,
                            readout_overlap: int = OVERLAP_AUTO) -> Tuple[torch.Tensor, torch.Tensor]:
    """Chunk-wise OSR forward.  Returns (y [B,T,H,d], state_out [B,H,m,d]).
    linearisation: LIN2 (default, eq. recurrence_linear2) or LIN1.
    schedule / chain_pairs / chain_wgs / readout_overlap: the matrix-core
    schedule (speed only)."""
    lib = load_library()
    desc = _desc_from(q, k, v, gamma, mu, state_in, y_dtype, mode, linearisation, schedule, chain_pairs, chain_wgs,
                      readout_overlap)
    _check_outputs(desc, q, state_in, state_out, y, y_dtype)
    st = _launch_stream(stream)
    with torch.cuda.stream(st):
        state_out, y = _outputs(desc, q, state_in, state_out, y, y_dtype)
        need = lattice_osr_workspace_bytes(desc, chunk_size)
        workspace, wbytes = _workspace(workspace, need, q.device)
        rc = lib.lattice_osr_fwd_chunked(ctypes.byref(desc), int(chunk_size), _ptr(q), _ptr(k), _ptr(v),
                                         _ptr(gamma), _ptr(mu), _ptr(state_in), _ptr(state_out), _ptr(y),
                                         _ptr(workspace), wbytes, st.cuda_stream)
    if rc != OK:
        raise OSRError(rc, "lattice_osr_fwd_chunked")
    return y, state_out


def lattice_osr_fwd_chunked_gated(q, k, v, gamma, mu, gate, state_in, chunk_size: int, *, mode: int = MODE_DEC,
                                  y_dtype=torch.float32, state_out=None, y=None, workspace=None, stream=None,
                                  linearisation: int = 0, schedule: int = SCHED_AUTO, chain_pairs: int = PAIRS_AUTO,
                                  chain_wgs: int = WGS_AUTO,
                                  readout_overlap: int = OVERLAP_AUTO) -> Tuple[torch.Tensor, torch.Tensor]:
    """Chunk-wise OSR forward with the GeLU post-gate fused into the output:
    y = OSR(...) * GeLU(gate), gate [B,T,H,d] in the inputs' dtype.
    Returns (y, state_out)."""
    lib = load_library()
    desc = _desc_from(q, k, v, gamma, mu, state_in, y_dtype, mode, linearisation, schedule, chain_pairs, chain_wgs,
                      readout_overlap)
    _check_tensor("gate", gate, tuple(v.shape), q.dtype, q.device)
    _check_outputs(desc, q, state_in, state_out, y, y_dtype)
    st = _launch_stream(stream)
    with torch.cuda.stream(st):
        state_out, y = _outputs(desc, q, state_in, state_out, y, y_dtype)
        need = lattice_osr_workspace_bytes(desc, chunk_size)
        workspace, wbytes = _workspace(workspace, need, q.device)
        rc = lib.lattice_osr_fwd_chunked_gated(ctypes.byref(desc), int(chunk_size), _ptr(q), _ptr(k), _ptr(v),
                                               _ptr(gamma), _ptr(mu), _ptr(gate), _ptr(state_in), _ptr(state_out),
                                               _ptr(y), _ptr(workspace), wbytes, st.cuda_stream)
    if rc != OK:
        raise OSRError(rc, "lattice_osr_fwd_chunked_gated")
    return y, state_out


def lattice_osr_fwd_chunked_noalloc(q, k, v, gamma, mu, state_in, chunk_size: int, *, state_out, y,
                                    mode: int = MODE_DEC, stream=None, linearisation: int = 0,
                                    schedule: int = SCHED_AUTO, chain_pairs: int = PAIRS_AUTO,
                                    chain_wgs: int = WGS_AUTO) -> Tuple[torch.Tensor, torch.Tensor]:
    """lattice_osr_fwd_chunked without a workspace: the library's per-GPU
    scratch holds it (at most NOALLOC_SCRATCH_BYTES).  The caller passes the
    outputs (y with y's dtype, state_out); nothing is allocated.  Calls that
    overlap on one GPU race on the scratch.  The read-out never overlaps
    here (all work on the one stream)."""
    lib = load_library()
    desc = _desc_from(q, k, v, gamma, mu, state_in, y.dtype, mode, linearisation, schedule, chain_pairs, chain_wgs)
    _check_outputs(desc, q, state_in, state_out, y, y.dtype)
    st = _launch_stream(stream)
    rc = lib.lattice_osr_fwd_chunked_noalloc(ctypes.byref(desc), int(chunk_size), _ptr(q), _ptr(k), _ptr(v),
                                             _ptr(gamma), _ptr(mu), _ptr(state_in), _ptr(state_out), _ptr(y),
                                             st.cuda_stream)
    if rc != OK:
        raise OSRError(rc, "lattice_osr_fwd_chunked_noalloc")
    return y, state_out


def lattice_osr_fwd_recurrent(q, k, v, gamma, mu, state_in, *, mode: int = MODE_DEC,
                              y_dtype=torch.float32, state_out=None, y=None,
                              stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Exact token-by-token OSR forward.  Returns (y, state_out)."""
    lib = load_library()
    desc = _desc_from(q, k, v, gamma, mu, state_in, y_dtype, mode)
    _check_outputs(desc, q, state_in, state_out, y, y_dtype)
    st = _launch_stream(stream)
    with torch.cuda.stream(st):
        state_out, y = _outputs(desc, q, state_in, state_out, y, y_dtype)
        rc = lib.lattice_osr_fwd_recurrent(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(gamma),
                                           _ptr(mu), _ptr(state_in), _ptr(state_out), _ptr(y), None, 0,
                                           st.cuda_stream)
    if rc != OK:
        raise OSRError(rc, "lattice_osr_fwd_recurrent")
    return y, state_out


def lattice_osr_decode_step(q, k, v, gamma, mu, state_in, *, mode: int = MODE_DEC,
                            y_dtype=torch.float32, state_out=None, y=None,
                            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One exact decode step (T = 1); state_out may be state_in (in place)."""
    lib = load_library()
    desc = _desc_from(q, k, v, gamma, mu, state_in, y_dtype, mode)
    _check_outputs(desc, q, state_in, state_out, y, y_dtype)
    st = _launch_stream(stream)
    with torch.cuda.stream(st):
        state_out, y = _outputs(desc, q, state_in, state_out, y, y_dtype)
        rc = lib.lattice_osr_decode_step(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(gamma),
                                         _ptr(mu), _ptr(state_in), _ptr(state_out), _ptr(y), None, 0,
                                         st.cuda_stream)
    if rc != OK:
        raise OSRError(rc, "lattice_osr_decode_step")
    return y, state_out


def lattice_osr_bwd_workspace_bytes(desc: lattice_osr_desc, chunk_size: int) -> int:
    n = int(load_library().lattice_osr_bwd_workspace_bytes(ctypes.byref(desc), int(chunk_size)))
    if n == ctypes.c_size_t(-1).value:
        raise OSRError(ERR_UNSUPPORTED, "lattice_osr_bwd_workspace_bytes")
    return n


def lattice_osr_bwd_chunked(q, k, v, gamma, mu, state_in, dy, dstate_out, chunk_size: int, *,
                            mode: int = MODE_DEC, grads: Optional[dict] = None, workspace=None,
                            stream=None, linearisation: int = LIN2, chain_wgs: int = WGS_AUTO,
                            bwd_form: int = BWD_AUTO) -> dict:
    """Backward of the chunk-wise forward: gradients of sum(dy*y) +
    sum(dstate_out*state_out) with respect to q, k, v, gamma, mu and
    state_in.  dy has y's shape (float32 or bfloat16), dstate_out the state's.
    Returns a dict of float32 tensors dq, dk, dv, dgamma, dmu, dstate_in
    (allocated unless passed in `grads`).  chain_wgs: WGS_ONE keeps each
    sequence of the token walk on one workgroup (speed only); bwd_form:
    BWD_WALK / BWD_CHUNK pick the backward's form (BWD_AUTO: the chunk form
    where it is built)."""
    return _bwd("lattice_osr_bwd_chunked", q, k, v, gamma, mu, state_in, dy, dstate_out, chunk_size, mode, grads,
                workspace, stream, linearisation, chain_wgs, bwd_form)


def lattice_osr_fwd_chunked_save(q, k, v, gamma, mu, state_in, chunk_size: int, *, mode: int = MODE_DEC,
                                 y_dtype=torch.float32, state_out=None, y=None, saved=None, stream=None,
                                 chain_wgs: int = WGS_AUTO, linearisation: int = LIN2):
    """The chunk-wise forward (small-chunk backward form only: C in 1, 2, 4, 8)
    that also stores what lattice_osr_bwd_chunked_saved needs.  Returns (y,
    state_out, saved); saved is a uint8 tensor of
    lattice_osr_bwd_workspace_bytes bytes (allocated unless passed), to be
    passed as that call's `saved`."""
    lib = load_library()
    desc = _desc_from(q, k, v, gamma, mu, state_in, y_dtype, mode, linearisation, chain_wgs=chain_wgs)
    _check_outputs(desc, q, state_in, state_out, y, y_dtype)
    st = _launch_stream(stream)
    with torch.cuda.stream(st):
        state_out, y = _outputs(desc, q, state_in, state_out, y, y_dtype)
        need = lattice_osr_bwd_workspace_bytes(desc, chunk_size)
        saved, sbytes = _workspace(saved, need, q.device)
        rc = lib.lattice_osr_fwd_chunked_save(ctypes.byref(desc), int(chunk_size), _ptr(q), _ptr(k), _ptr(v),
                                              _ptr(gamma), _ptr(mu), _ptr(state_in), _ptr(state_out), _ptr(y),
                                              _ptr(saved), sbytes, st.cuda_stream)
    if rc != OK:
        raise OSRError(rc, "lattice_osr_fwd_chunked_save")
    return y, state_out, saved


def lattice_osr_bwd_chunked_saved(q, k, v, gamma, mu, state_in, dy, dstate_out, chunk_size: int, *, saved,
                                  mode: int = MODE_DEC, grads: Optional[dict] = None, stream=None,
                                  chain_wgs: int = WGS_AUTO, linearisation: int = LIN2) -> dict:
    """lattice_osr_bwd_chunked's gradients, bit for bit, from the values a
    lattice_osr_fwd_chunked_save call with the same inputs stored in `saved`
    (its forward pass skipped)."""
    if saved is None:
        raise ValueError("saved: the tensor lattice_osr_fwd_chunked_save returned")
    return _bwd("lattice_osr_bwd_chunked_saved", q, k, v, gamma, mu, state_in, dy, dstate_out, chunk_size, mode,
                grads, saved, stream, linearisation, chain_wgs, BWD_AUTO)


def _bwd(entry, q, k, v, gamma, mu, state_in, dy, dstate_out, chunk_size, mode, grads, workspace, stream,
         linearisation, chain_wgs, bwd_form) -> dict:
    lib = load_library()
    desc = _desc_from(q, k, v, gamma, mu, state_in, dy.dtype, mode, linearisation, chain_wgs=chain_wgs,
                      bwd_form=bwd_form)
    _check_tensor("dy", dy, tuple(v.shape), None, q.device)
    _check_tensor("dstate_out", dstate_out, tuple(state_in.shape), torch.float32, q.device)
    named = (("q", q), ("k", k), ("v", v), ("gamma", gamma), ("mu", mu), ("state_in", state_in))
    if grads is not None:
        for n, t in named:
            if "d" + n not in grads:
                raise ValueError(f"grads lacks d{n}")
            _check_tensor("d" + n, grads["d" + n], tuple(t.shape), torch.float32, q.device)
    _check_cuda(q)
    st = _launch_stream(stream)
    with torch.cuda.stream(st):
        if grads is None:
            grads = {"d" + n: torch.empty(t.shape, dtype=torch.float32, device=q.device) for n, t in named}
        need = lattice_osr_bwd_workspace_bytes(desc, chunk_size)
        workspace, wbytes = _workspace(workspace, need, q.device)
        g = grads
        rc = getattr(lib, entry)(ctypes.byref(desc), int(chunk_size), _ptr(q), _ptr(k), _ptr(v),
                                 _ptr(gamma), _ptr(mu), _ptr(state_in), _ptr(dy), _ptr(dstate_out),
                                 _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dgamma"]),
                                 _ptr(g["dmu"]), _ptr(g["dstate_in"]), _ptr(workspace), wbytes,
                                 st.cuda_stream)
    if rc != OK:
        raise OSRError(rc, entry)
    return grads


# ------------------------------------------------------------ layer glue --
def lattice_osr_glue_pre(xq, xk, gamma_logit, conv_wq, conv_wk, conv_bq=None, conv_bk=None, hist_q=None,
                         hist_k=None, *, q=None, k=None, gamma=None, hist_q_out=None, hist_k_out=None,
                         return_history: bool = False, stream=None):
    """q = conv4(xq), k = conv4(xk), gamma = sigmoid(gamma_logit) in one pass.

    xq, xk [B,T,H,m] and gamma_logit [B,T,H,m] or [B,T,H] share a dtype (float32 or
    bfloat16); conv_w* [H,m,4] and conv_b* [H,m] are float32; hist_* [B,3,H,m] carry
    the three raw rows before this call.  Returns (q, k, gamma) and, with
    return_history, also the history for the next call."""
    lib = load_library()
    if xq.dim() != 4 or xq.dtype not in _DT:
        raise ValueError("xq/xk are [B,T,H,m] float32 or bfloat16")
    B, T, H, m = xq.shape
    dev = xq.device
    per_slot = 1 if gamma_logit.dim() == 4 else 0
    gshape = (B, T, H, m) if per_slot else (B, T, H)
    _check_tensor("xq", xq, (B, T, H, m), xq.dtype)
    _check_tensor("xk", xk, (B, T, H, m), xq.dtype, dev)
    _check_tensor("gamma_logit", gamma_logit, gshape, xq.dtype, dev)
    _check_tensor("conv_wq", conv_wq, (H, m, 4), torch.float32, dev)
    _check_tensor("conv_wk", conv_wk, (H, m, 4), torch.float32, dev)
    for name, t in (("conv_bq", conv_bq), ("conv_bk", conv_bk)):
        if t is not None:
            _check_tensor(name, t, (H, m), torch.float32, dev)
    if (hist_q is None) != (hist_k is None):
        raise ValueError("pass both histories or neither")
    for name, t in (("hist_q", hist_q), ("hist_k", hist_k)):
        if t is not None:
            _check_tensor(name, t, (B, 3, H, m), xq.dtype, dev)
    _check_cuda(xq)
    desc = make_desc(B, T, H, m, m, per_slot, _DT[xq.dtype], F32)
    st = _launch_stream(stream)
    with torch.cuda.stream(st):
        outs = {}
        for name, t, like, shape in (("q", q, xq, (B, T, H, m)), ("k", k, xk, (B, T, H, m)),
                                     ("gamma", gamma, gamma_logit, gshape)):
            if t is None:
                t = torch.empty_like(like)
            else:
                _check_tensor(name, t, shape, xq.dtype, dev)
            outs[name] = t
        q, k, gamma = outs["q"], outs["k"], outs["gamma"]
        if return_history:
            hist_q_out = xq.new_empty((B, 3, H, m)) if hist_q_out is None else hist_q_out
            hist_k_out = xk.new_empty((B, 3, H, m)) if hist_k_out is None else hist_k_out
        for name, t in (("hist_q_out", hist_q_out), ("hist_k_out", hist_k_out)):
            if t is not None:
                _check_tensor(name, t, (B, 3, H, m), xq.dtype, dev)
        rc = lib.lattice_osr_glue_pre(ctypes.byref(desc), _ptr(xq), _ptr(xk), _ptr(gamma_logit), _ptr(conv_wq),
                                      _ptr(conv_wk), _ptr(conv_bq), _ptr(conv_bk), _ptr(hist_q), _ptr(hist_k),
                                      _ptr(q), _ptr(k), _ptr(gamma), _ptr(hist_q_out), _ptr(hist_k_out),
                                      st.cuda_stream)
    if rc != OK:
        raise OSRError(rc, "lattice_osr_glue_pre")
    if return_history:
        return q, k, gamma, hist_q_out, hist_k_out
    return q, k, gamma


def lattice_osr_glue_post(y, gate, *, out=None, stream=None):
    """out = y * GeLU(gate) (exact GeLU); y [B,T,H,d] float32 or bfloat16, gate of y's shape in
    float32 or bfloat16.  out may be y (in place)."""
    lib = load_library()
    if y.dim() != 4 or y.dtype not in _DT or gate.dtype not in _DT:
        raise ValueError("y and gate are [B,T,H,d] float32 or bfloat16 tensors of one shape")
    _check_tensor("y", y, tuple(y.shape), y.dtype)
    _check_tensor("gate", gate, tuple(y.shape), gate.dtype, y.device)
    _check_cuda(y)
    B, T, H, d = y.shape
    desc = make_desc(B, T, H, 16, d, 1, _DT[gate.dtype], _DT[y.dtype])
    st = _launch_stream(stream)
    with torch.cuda.stream(st):
        if out is None:
            out = torch.empty_like(y)
        else:
            _check_tensor("out", out, tuple(y.shape), y.dtype, y.device)
        rc = lib.lattice_osr_glue_post(ctypes.byref(desc), _ptr(y), _ptr(gate), _ptr(out), st.cuda_stream)
    if rc != OK:
        raise OSRError(rc, "lattice_osr_glue_post")
    return out


# ---------------------------------------- element-wise gated recurrence --
def _on(device, stream, fn):
    """fn(stream handle) with the tensors' device current and, where a stream
    is given, under it, so that what fn allocates follows its order."""
    if stream is None and device.index == torch.cuda.current_device():
        # the handle alone: a Stream object costs 2.7 us, of the 10 of a one-token call
        return fn(torch._C._cuda_getCurrentRawStream(device.index))
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    with torch.cuda.device(device):
        st = torch.cuda.current_stream() if stream is None else stream
        with torch.cuda.stream(st):
            return fn(st.cuda_stream)


def _query(fn, desc):
    """What the library answers for a size; None for a descriptor that it refuses."""
    n = int(getattr(load_library(), fn)(ctypes.byref(desc)))
    return None if n == ctypes.c_size_t(-1).value else n


def _bytes_of(fn, desc):
    n = _query(fn, desc)
    if n is None:
        raise OSRError(ERR_SHAPE, fn)
    return n


def make_scan_desc(B, T, D, in_dtype=BF16, y_dtype=F32, grad_dtype=F32, input_weight=SCAN_COMPLEMENT):
    return lattice_osr_scan_desc(B, T, D, in_dtype, y_dtype, grad_dtype, input_weight)


@functools.lru_cache(maxsize=1024)
def _scan_sizes(fields):
    """(saved, workspace) bytes of a scan descriptor, given its fields; zeros for one that the call
    itself refuses, with its status."""
    desc = lattice_osr_scan_desc(*fields)
    return (_query("lattice_osr_scan_saved_bytes", desc) or 0, _query("lattice_osr_scan_workspace_bytes", desc) or 0)


@functools.lru_cache(maxsize=1024)
def _norm_size(fields):
    """Workspace bytes of a norm descriptor's backward, given its fields; 0 as above."""
    return _query("lattice_osr_norm_bwd_workspace_bytes", lattice_osr_norm_desc(*fields)) or 0


def lattice_osr_scan_saved_bytes(desc: lattice_osr_scan_desc) -> int:
    return _bytes_of("lattice_osr_scan_saved_bytes", desc)


def lattice_osr_scan_workspace_bytes(desc: lattice_osr_scan_desc) -> int:
    return _bytes_of("lattice_osr_scan_workspace_bytes", desc)


def _scan_desc(v, mu_logit, gamma_logit, lengths, y_dtype, grad_dtype, input_weight):
    """Descriptor fields of a scan call, after checking every input against them: v,
    mu_logit, gamma_logit [B,T,D] or [B,T,H,d] in one dtype, lengths [B] int32;
    all contiguous, on one GPU.  Returns them with the states' shape."""
    if v.dim() not in (3, 4):
        raise ValueError("v/mu_logit/gamma_logit are [B,T,D] or [B,T,H,d]")
    if v.dtype not in _DT:
        raise ValueError("inputs must be float32 or bfloat16")
    if y_dtype not in _DT or grad_dtype not in _DT:
        raise ValueError("y_dtype and grad_dtype must be torch.float32 or torch.bfloat16")
    shape, dev = v.shape, v.device
    _check_tensor("v", v, shape, None)
    _check_tensor("mu_logit", mu_logit, shape, v.dtype, dev)
    if gamma_logit is not None:
        _check_tensor("gamma_logit", gamma_logit, shape, v.dtype, dev)
    if lengths is not None:
        _check_tensor("lengths", lengths, (shape[0],), torch.int32, dev)
    D = shape[2] if len(shape) == 3 else shape[2] * shape[3]
    if max(shape[0], shape[1], D) > 2 ** 31 - 1:
        raise ValueError(f"shape {tuple(shape)}: sizes are at most 2^31 - 1")
    fields = (shape[0], shape[1], D, _DT[v.dtype], _DT[y_dtype], _DT[grad_dtype], input_weight)
    return fields, (shape[0], *shape[2:])


def _room(t, need, lead):
    """(the caller's buffer or a new one of `need` bytes beside lead, its bytes); (None, 0) where neither is."""
    if t is not None:
        return _workspace(t, need, lead.device)
    return (lead.new_empty(need, dtype=torch.uint8), need) if need else (None, 0)


def lattice_osr_scan_fwd(v, mu_logit, state_in=None, *, gamma_logit=None, lengths=None,
                         input_weight: int = SCAN_COMPLEMENT, y_dtype=torch.float32, y=None, state_out=None,
                         save: bool = False, saved=None, workspace=None, stream=None):
    """h_t = mu_t h_{t-1} + w(mu_t) gamma_t v_t with mu = sigmoid(mu_logit) and
    gamma = sigmoid(gamma_logit) (1 without it), y = h; w by input_weight: 1,
    1 - mu or sqrt(1 - mu^2).

    v, mu_logit, gamma_logit [B,T,D] or [B,T,H,d] share a dtype (float32 or bfloat16);
    state_in (None: zeros) and state_out are [B,D] or [B,H,d] float32, state_out may
    be state_in; lengths [B] int32: the tokens of each sequence, y is zero behind them.
    Returns (y, state_out) and, with save (or `saved`, a uint8 tensor of
    lattice_osr_scan_saved_bytes), what lattice_osr_scan_bwd needs."""
    lib = load_library()
    fields, sshape = _scan_desc(v, mu_logit, gamma_logit, lengths, y_dtype, torch.float32, input_weight)
    dev = v.device
    for name, t in (("state_in", state_in), ("state_out", state_out)):
        if t is not None:
            _check_tensor(name, t, sshape, torch.float32, dev)
    if y is not None:
        _check_tensor("y", y, v.shape, y_dtype, dev)
    _check_cuda(v)
    save = save or saved is not None

    def call(st):
        yy = torch.empty_like(v, dtype=y_dtype) if y is None else y
        so = v.new_empty(sshape, dtype=torch.float32) if state_out is None else state_out
        snb, wnb = _scan_sizes(fields)
        sv, sbytes = _room(saved, snb, v) if save else (None, 0)
        ws, wbytes = _room(workspace, wnb, v)
        desc = lattice_osr_scan_desc(*fields)
        rc = lib.lattice_osr_scan_fwd(ctypes.byref(desc), _ptr(v), _ptr(mu_logit), _ptr(gamma_logit), _ptr(lengths),
                                      _ptr(state_in), _ptr(so), _ptr(yy), _ptr(sv), sbytes, _ptr(ws), wbytes, st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_scan_fwd")
        return (yy, so, sv) if save else (yy, so)

    return _on(dev, stream, call)


def lattice_osr_scan_bwd(v, mu_logit, dy, dstate_out=None, *, saved, gamma_logit=None, lengths=None,
                         input_weight: int = SCAN_COMPLEMENT, grad_dtype=torch.float32, grads: Optional[dict] = None,
                         workspace=None, stream=None) -> dict:
    """Gradients of sum(dy*y) + sum(dstate_out*state_out) of lattice_osr_scan_fwd with
    the same inputs, whose `saved` this call takes.  dy has v's shape (float32 or
    bfloat16), dstate_out the state's (None: zeros).  Returns a dict of dv, dmu_logit
    (and dgamma_logit, with gamma_logit) in grad_dtype and dstate_in in float32,
    allocated unless passed in `grads`."""
    lib = load_library()
    if saved is None:
        raise ValueError("saved: the tensor lattice_osr_scan_fwd returned with save=True")
    fields, sshape = _scan_desc(v, mu_logit, gamma_logit, lengths, dy.dtype, grad_dtype, input_weight)
    dev = v.device
    _check_tensor("dy", dy, v.shape, None, dev)
    if dstate_out is not None:
        _check_tensor("dstate_out", dstate_out, sshape, torch.float32, dev)
    want = [("dv", v, v.shape, grad_dtype), ("dmu_logit", v, v.shape, grad_dtype)]
    if gamma_logit is not None:
        want.append(("dgamma_logit", v, v.shape, grad_dtype))
    want.append(("dstate_in", dstate_out, sshape, torch.float32))
    _check_grads(grads, want, dev)
    _check_cuda(v)

    def call(st):
        g = _grads(grads, want, v)
        sv, sbytes = _workspace(saved, 0, dev)
        ws, wbytes = _room(workspace, _scan_sizes(fields)[1], v)
        desc = lattice_osr_scan_desc(*fields)
        rc = lib.lattice_osr_scan_bwd(ctypes.byref(desc), _ptr(v), _ptr(mu_logit), _ptr(gamma_logit), _ptr(lengths),
                                      _ptr(sv), sbytes, _ptr(dy), _ptr(dstate_out), _ptr(g["dv"]),
                                      _ptr(g["dmu_logit"]), _ptr(g.get("dgamma_logit")), _ptr(g["dstate_in"]),
                                      _ptr(ws), wbytes, st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_scan_bwd")
        return g

    return _on(dev, stream, call)


def _check_grads(grads, want, dev):
    if grads is None:
        return
    for name, _, shape, dtype in want:
        if name not in grads:
            raise ValueError(f"grads lacks {name}")
        _check_tensor(name, grads[name], shape, dtype, dev)


def _grads(grads, want, lead):
    """The caller's gradients, or new ones on lead's device, each like the tensor it belongs to."""
    if grads is not None:
        return {name: grads[name] for name, *_ in want}
    return {name: lead.new_empty(shape, dtype=dtype) if like is None else torch.empty_like(like, dtype=dtype)
            for name, like, shape, dtype in want}


def lattice_osr_scan_step(v, mu_logit, state_in, *, gamma_logit=None, input_weight: int = SCAN_COMPLEMENT,
                          y_dtype=torch.float32, y=None, state_out=None, stream=None):
    """One token of lattice_osr_scan_fwd (T = 1) for every sequence; state_out
    may be state_in (in place).  Returns (y, state_out)."""
    lib = load_library()
    fields, sshape = _scan_desc(v, mu_logit, gamma_logit, None, y_dtype, torch.float32, input_weight)
    dev = v.device
    _check_tensor("state_in", state_in, sshape, torch.float32, dev)
    if state_out is not None:
        _check_tensor("state_out", state_out, sshape, torch.float32, dev)
    if y is not None:
        _check_tensor("y", y, v.shape, y_dtype, dev)
    _check_cuda(v)

    def call(st):
        yy = torch.empty_like(v, dtype=y_dtype) if y is None else y
        so = torch.empty_like(state_in) if state_out is None else state_out
        desc = lattice_osr_scan_desc(*fields)
        rc = lib.lattice_osr_scan_step(ctypes.byref(desc), _ptr(v), _ptr(mu_logit), _ptr(gamma_logit), _ptr(state_in),
                                       _ptr(so), _ptr(yy), st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_scan_step")
        return yy, so

    return _on(dev, stream, call)


# ------------------------------------------------- norms around a block --
def make_norm_desc(R, D, in_dtype=BF16, res_dtype=BF16, grad_dtype=F32, gate_kind=GATE_NONE, post_norm=1, pre_norm=1,
                   eps=1e-6):
    return lattice_osr_norm_desc(R, D, in_dtype, res_dtype, grad_dtype, gate_kind, post_norm, pre_norm, eps)


def lattice_osr_norm_bwd_workspace_bytes(desc: lattice_osr_norm_desc) -> int:
    return _bytes_of("lattice_osr_norm_bwd_workspace_bytes", desc)


def _norm_desc(y, x, gate, gate_kind, post_norm, w_post, scale, pre_norm, w_pre, eps, z_dtype, x_dtype, grad_dtype):
    """Descriptor fields of a norm call, after checking every input against them: rows
    [..., D] of y, gate (one dtype) and x, weights [D] float32; all contiguous,
    on one GPU."""
    lead = y if y is not None else x
    if lead is None:
        raise ValueError("pass y, x or both")
    if lead.dim() < 1:
        raise ValueError("y, x and gate are [..., D]")
    shape, dev = lead.shape, lead.device
    D = shape[-1]
    in_dtype = y.dtype if y is not None else z_dtype or x.dtype
    res_dtype = x.dtype if x is not None else x_dtype or in_dtype
    for dt in (in_dtype, res_dtype, grad_dtype):
        if dt not in _DT:
            raise ValueError("tensors must be float32 or bfloat16")
    if gate is None:
        gate_kind = GATE_NONE
    elif gate_kind == GATE_NONE:
        raise ValueError("gate given with GATE_NONE")
    for name, t, dt in (("y", y, in_dtype), ("x", x, res_dtype), ("gate", gate, in_dtype)):
        if t is not None:
            _check_tensor(name, t, shape, dt, dev)
    for name, t in (("w_post", w_post), ("scale", scale), ("w_pre", w_pre)):
        if t is not None:
            _check_tensor(name, t, (D,), torch.float32, dev)
    R = lead.numel() // D if D else 0
    if R > 2 ** 31 - 1:
        raise ValueError(f"{R} rows: at most 2^31 - 1")
    fields = (R, D, _DT[in_dtype], _DT[res_dtype], _DT[grad_dtype], gate_kind, int(post_norm and y is not None),
              int(pre_norm), eps)
    return fields, lead, in_dtype, res_dtype


def lattice_osr_norm_fwd(y=None, x=None, *, gate=None, gate_kind: int = GATE_GELU, post_norm: bool = True,
                         w_post=None, scale=None, pre_norm: bool = True, w_pre=None, eps: float = 1e-6,
                         z_dtype=None, x_dtype=None, x_out=None, z=None, stream=None):
    """u = y phi(gate), n = u / rms(u) w_post, x_out = x + scale n, z = x_out / rms(x_out) w_pre
    over the last dimension, rms(a) = sqrt(mean(a^2) + eps).

    y and gate [..., D] share a dtype, which is z's too; x [..., D] has its own (float32 or
    bfloat16 each); the weights are [D] float32, None: ones.  gate None: no gate; gate_kind
    GATE_GELU or GATE_SILU.  x None: no residual, x_out in x_dtype (y's dtype if None).  y None:
    only z = x / rms(x) w_pre, in z_dtype (x's dtype if None).  x_out may be x (in place).
    Returns (x_out, z); x_out is None without y, z without pre_norm."""
    lib = load_library()
    fields, lead, in_dtype, res_dtype = _norm_desc(y, x, gate, gate_kind, post_norm, w_post, scale, pre_norm, w_pre,
                                                 eps, z_dtype, x_dtype, torch.float32)
    dev = lead.device
    if z_dtype is not None and z_dtype != in_dtype:
        raise ValueError("z_dtype is y's dtype")
    if x_dtype is not None and x_dtype != res_dtype:
        raise ValueError("x_dtype is x's dtype")
    if x_out is not None:
        _check_tensor("x_out", x_out, lead.shape, res_dtype, dev)
    if z is not None:
        _check_tensor("z", z, lead.shape, in_dtype, dev)
    _check_cuda(lead)

    def call(st):
        xo = torch.empty_like(lead, dtype=res_dtype) if x_out is None and y is not None else x_out
        zz = torch.empty_like(lead, dtype=in_dtype) if z is None and pre_norm else z
        desc = lattice_osr_norm_desc(*fields)
        rc = lib.lattice_osr_norm_fwd(ctypes.byref(desc), _ptr(y), _ptr(gate), _ptr(x), _ptr(w_post), _ptr(scale),
                                      _ptr(w_pre), _ptr(xo), _ptr(zz), st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_norm_fwd")
        return xo, zz

    return _on(dev, stream, call)


def lattice_osr_norm_bwd(y=None, x=None, dx_out=None, dz=None, *, gate=None, gate_kind: int = GATE_GELU,
                         post_norm: bool = True, w_post=None, scale=None, pre_norm: bool = True, w_pre=None,
                         eps: float = 1e-6, grad_dtype=torch.float32, grads: Optional[dict] = None, workspace=None,
                         stream=None) -> dict:
    """Gradients of sum(dx_out*x_out) + sum(dz*z) of lattice_osr_norm_fwd with the same inputs.
    dx_out (x's dtype; None with pre_norm: zeros) and dz (y's dtype, with pre_norm) have y's shape.
    Returns a dict of dy, dgate (grad_dtype), dx (x's dtype) and dw_post, dscale, dw_pre (float32), each
    where its operand was passed, allocated unless passed in `grads` (dx may be dx_out)."""
    lib = load_library()
    fields, lead, in_dtype, res_dtype = _norm_desc(y, x, gate, gate_kind, post_norm, w_post, scale, pre_norm, w_pre,
                                                 eps, dz.dtype if dz is not None else None,
                                                 dx_out.dtype if dx_out is not None else None, grad_dtype)
    dev = lead.device
    for name, t, dt in (("dx_out", dx_out, res_dtype), ("dz", dz, in_dtype)):
        if t is not None:
            _check_tensor(name, t, lead.shape, dt, dev)
    f32 = torch.float32
    want = [(n, t, t.shape, dt) for n, t, dt in (("dy", y, grad_dtype), ("dgate", gate, grad_dtype),
                                                 ("dx", x, res_dtype), ("dw_post", w_post, f32),
                                                 ("dscale", scale, f32), ("dw_pre", w_pre, f32)) if t is not None]
    _check_grads(grads, want, dev)
    _check_cuda(lead)

    def call(st):
        g = _grads(grads, want, lead)
        sums = w_post is not None or scale is not None or w_pre is not None
        ws, wbytes = _room(workspace, _norm_size(fields) if sums else 0, lead)
        desc = lattice_osr_norm_desc(*fields)
        rc = lib.lattice_osr_norm_bwd(ctypes.byref(desc), _ptr(y), _ptr(gate), _ptr(x), _ptr(w_post), _ptr(scale),
                                      _ptr(w_pre), _ptr(dx_out), _ptr(dz), _ptr(g.get("dy")), _ptr(g.get("dgate")),
                                      _ptr(g.get("dx")), _ptr(g.get("dw_post")), _ptr(g.get("dscale")),
                                      _ptr(g.get("dw_pre")), _ptr(ws), wbytes, st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_norm_bwd")
        return g

    return _on(dev, stream, call)


# -------------------------------------- selective state space layer --
def _row(name, t, shape, dtype, dev, inner):
    """Elements from one token's row of t to the next (0: contiguous), after checking its shape, dtype and
    device: t is [B,T,...] whose last `inner` dimensions are contiguous and whose rows
    are one stride apart, as a slice of the last dimension of a contiguous tensor is.  (The library takes strides of
    up to 2^22 elements; one token of each of several long sequences can lie further apart, and has to be copied.)"""
    if t.is_contiguous():
        if t.shape == shape and t.dtype is dtype and t.device == dev:
            return 0
        _check_tensor(name, t, shape, dtype, dev)
        return 0
    if tuple(t.shape) != tuple(shape):
        _shape_error(name, t, shape)
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    width = 1
    for k in range(t.dim() - 1, t.dim() - 1 - inner, -1):
        if t.shape[k] != 1 and t.stride(k) != width:
            raise ValueError(f"{name} must be contiguous but for the stride between tokens")
        width *= t.shape[k]
    B, T = t.shape[:2]
    row = t.stride(1) if T > 1 else t.stride(0)
    if B > 1 and t.stride(0) != T * row or not width <= row < 2 ** 31:
        raise ValueError(f"{name} must be contiguous but for the stride between tokens")
    return row


def _lead(name, x):
    """(B, T, D, shape of one token) of a [B,T,D] or [B,T,H,d] tensor."""
    if x.dim() not in (3, 4):
        raise ValueError(f"{name} is [B,T,D] or [B,T,H,d]")
    if x.dtype not in _DT:
        raise ValueError("inputs must be float32 or bfloat16")
    B, T, *tok = x.shape
    D = tok[0] if len(tok) == 1 else tok[0] * tok[1]
    if B > 2 ** 31 - 1 or T > 2 ** 31 - 1 or D > 2 ** 31 - 1:
        raise ValueError(f"shape {tuple(x.shape)}: sizes are at most 2^31 - 1")
    return B, T, D, tuple(tok)


def _check_tokens(lengths, segments, B, T, dev):
    if lengths is not None:
        _check_tensor("lengths", lengths, (B,), torch.int32, dev)
    if segments is not None:
        _check_tensor("segments", segments, (B, T), torch.int32, dev)


def _check_dtypes(*dtypes):
    for dt in dtypes:
        if dt not in _DT:
            raise ValueError("tensors must be float32 or bfloat16")


@functools.lru_cache(maxsize=1024)
def _ref(kind, fields):
    """A reference to the descriptor of these fields, which the library only reads."""
    return ctypes.byref(kind(*fields))


def make_conv_desc(B, T, D, W, act=CONV_SILU, in_dtype=BF16, y_dtype=BF16, grad_dtype=F32, x_row=0):
    return lattice_osr_conv_desc(B, T, D, W, act, in_dtype, y_dtype, grad_dtype, x_row)


def lattice_osr_conv_bwd_workspace_bytes(desc: lattice_osr_conv_desc) -> int:
    return _bytes_of("lattice_osr_conv_bwd_workspace_bytes", desc)


def _conv_desc(x, w, bias, hist_in, act, lengths, segments, y_dtype, grad_dtype):
    """Descriptor fields of a convolution call, after checking every input against them."""
    B, T, D, tok = _lead("x", x)
    _check_dtypes(y_dtype, grad_dtype)
    dev = x.device
    if w.dim() != x.dim() - 1:
        raise ValueError("w is [D,W], or [H,d,W] beside x [B,T,H,d]")
    W = w.shape[-1]
    _check_tensor("w", w, tok + (W,), torch.float32, dev)
    if bias is not None:
        _check_tensor("bias", bias, tok, torch.float32, dev)
    row = 0 if x.is_contiguous() else _row("x", x, x.shape, None, None, len(tok))
    hshape = (B, W - 1) + tok
    if hist_in is not None:
        _check_tensor("hist_in", hist_in, hshape, x.dtype, dev)
    _check_tokens(lengths, segments, B, T, dev)
    return (B, T, D, W, act, _DT[x.dtype], _DT[y_dtype], _DT[grad_dtype], row), hshape


def lattice_osr_conv_fwd(x, w, bias=None, hist_in=None, *, act: int = CONV_SILU, lengths=None, segments=None,
                         y_dtype=None, y=None, hist_out=None, return_history: bool = False, stream=None):
    """p_t = bias + sum_j w[j] x_{t-W+1+j} per channel, y = p sigmoid(p) (act CONV_SILU) or p (CONV_NONE).

    x [B,T,D] or [B,T,H,d] (float32 or bfloat16; its rows may be a stride of up to 2^22 elements apart, as in a slice of
    a projection's output), w [D,W] and bias [D] float32; hist_in [B,W-1,D] in x's dtype, the raw rows before
    the first token (None: zeros); lengths [B] int32: the tokens of each sequence, y is zero behind them; segments
    [B,T] int32: the document of every token, whose border no tap crosses.  y has x's shape, in y_dtype (x's
    dtype if None).  Returns y and, with return_history (or `hist_out`), the raw rows behind the last
    token, for the next call."""
    lib = load_library()
    y_dtype = x.dtype if y_dtype is None else y_dtype
    fields, hshape = _conv_desc(x, w, bias, hist_in, act, lengths, segments, y_dtype, torch.float32)
    dev = x.device
    if y is not None:
        _check_tensor("y", y, x.shape, y_dtype, dev)
    if hist_out is not None:
        _check_tensor("hist_out", hist_out, hshape, x.dtype, dev)
    _check_cuda(x)
    history = return_history or hist_out is not None

    def call(st):
        yy = x.new_empty(x.shape, dtype=y_dtype) if y is None else y
        ho = x.new_empty(hshape) if hist_out is None and history else hist_out
        rc = lib.lattice_osr_conv_fwd(_ref(lattice_osr_conv_desc, fields), _ptr(x), _ptr(w), _ptr(bias), _ptr(lengths),
                                      _ptr(segments), _ptr(hist_in), _ptr(ho), _ptr(yy), st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_conv_fwd")
        return (yy, ho) if history else yy

    return _on(dev, stream, call)


@functools.lru_cache(maxsize=1024)
def _conv_size(fields):
    return _query("lattice_osr_conv_bwd_workspace_bytes", lattice_osr_conv_desc(*fields)) or 0


def lattice_osr_conv_bwd(x, w, dy, bias=None, hist_in=None, dhist_out=None, *, act: int = CONV_SILU, lengths=None,
                         segments=None, grad_dtype=torch.float32, grads: Optional[dict] = None, workspace=None,
                         stream=None) -> dict:
    """Gradients of sum(dy*y) + sum(dhist_out*hist_out) of lattice_osr_conv_fwd with the same inputs.  dy has
    x's shape (float32 or bfloat16), dhist_out the history's in grad_dtype (None: zeros).  Returns a dict of dx,
    dhist_in (grad_dtype; the latter with hist_in), dw and dbias (float32; the latter with bias), allocated
    unless passed in `grads`."""
    lib = load_library()
    fields, hshape = _conv_desc(x, w, bias, hist_in, act, lengths, segments, dy.dtype, grad_dtype)
    dev = x.device
    _check_tensor("dy", dy, x.shape, None, dev)
    if dhist_out is not None:
        _check_tensor("dhist_out", dhist_out, hshape, grad_dtype, dev)
    f32 = torch.float32
    want = [("dx", None, x.shape, grad_dtype), ("dw", None, w.shape, f32)]
    if bias is not None:
        want.append(("dbias", None, bias.shape, f32))
    if hist_in is not None:
        want.append(("dhist_in", None, hshape, grad_dtype))
    _check_grads(grads, want, dev)
    _check_cuda(x)

    def call(st):
        g = _grads(grads, want, x)
        ws, wbytes = _room(workspace, _conv_size(fields), x)
        rc = lib.lattice_osr_conv_bwd(_ref(lattice_osr_conv_desc, fields), _ptr(x), _ptr(w), _ptr(bias), _ptr(lengths),
                                      _ptr(segments), _ptr(hist_in), _ptr(dy), _ptr(dhist_out), _ptr(g["dx"]),
                                      _ptr(g["dw"]), _ptr(g.get("dbias")), _ptr(g.get("dhist_in")), _ptr(ws), wbytes,
                                      st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_conv_bwd")
        return g

    return _on(dev, stream, call)


def lattice_osr_conv_step(x, w, hist_in, bias=None, *, act: int = CONV_SILU, y_dtype=None, y=None, hist_out=None,
                          stream=None):
    """One token of lattice_osr_conv_fwd (T = 1) for every sequence; hist_out may be hist_in (in place).
    Returns (y, hist_out)."""
    lib = load_library()
    y_dtype = x.dtype if y_dtype is None else y_dtype
    if hist_in is None:
        raise ValueError("hist_in: the history of every sequence (zeros at its start)")
    fields, hshape = _conv_desc(x, w, bias, hist_in, act, None, None, y_dtype, torch.float32)
    dev = x.device
    if y is not None:
        _check_tensor("y", y, x.shape, y_dtype, dev)
    if hist_out is not None:
        _check_tensor("hist_out", hist_out, hshape, x.dtype, dev)
    _check_cuda(x)

    def call(st):
        yy = x.new_empty(x.shape, dtype=y_dtype) if y is None else y
        ho = torch.empty_like(hist_in) if hist_out is None else hist_out
        rc = lib.lattice_osr_conv_step(_ref(lattice_osr_conv_desc, fields), _ptr(x), _ptr(w), _ptr(bias),
                                       _ptr(hist_in), _ptr(ho), _ptr(yy), st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_conv_step")
        return yy, ho

    return _on(dev, stream, call)


def make_ssm_desc(B, T, D, N, G=1, in_dtype=BF16, y_dtype=BF16, grad_dtype=F32, softplus=1, x_row=0, dt_row=0, z_row=0,
                  b_row=0, c_row=0):
    return lattice_osr_ssm_desc(B, T, D, N, G, in_dtype, y_dtype, grad_dtype, softplus, x_row, dt_row, z_row, b_row,
                                c_row)


def lattice_osr_ssm_saved_bytes(desc: lattice_osr_ssm_desc) -> int:
    return _bytes_of("lattice_osr_ssm_saved_bytes", desc)


def lattice_osr_ssm_workspace_bytes(desc: lattice_osr_ssm_desc) -> int:
    return _bytes_of("lattice_osr_ssm_workspace_bytes", desc)


def lattice_osr_ssm_bwd_workspace_bytes(desc: lattice_osr_ssm_desc) -> int:
    return _bytes_of("lattice_osr_ssm_bwd_workspace_bytes", desc)


@functools.lru_cache(maxsize=1024)
def _ssm_sizes(fields):
    """(saved, forward's workspace, backward's workspace) bytes; zeros for a descriptor that the call itself
    refuses, with its status."""
    desc = lattice_osr_ssm_desc(*fields)
    return tuple(_query("lattice_osr_ssm_" + f, desc) or 0 for f in ("saved_bytes", "workspace_bytes",
                                                                    "bwd_workspace_bytes"))


def _ssm_desc(x, dt, A, B, C, D, z, dt_bias, softplus, lengths, segments, y_dtype, grad_dtype):
    """Descriptor fields of a state space call and its state's shape, after checking every input against them."""
    nb, T, ch, tok = _lead("x", x)
    _check_dtypes(y_dtype, grad_dtype)
    dev, dtype = x.device, x.dtype
    if A.dim() != x.dim() - 1:
        raise ValueError("A is [D,N], or [H,d,N] beside x [B,T,H,d]")
    N = A.shape[-1]
    _check_tensor("A", A, tok + (N,), torch.float32, dev)
    for name, t in (("D", D), ("dt_bias", dt_bias)):
        if t is not None:
            _check_tensor(name, t, tok, torch.float32, dev)
    k = len(tok)
    rows = [0 if x.is_contiguous() else _row("x", x, x.shape, None, None, k), _row("dt", dt, x.shape, dtype, dev, k),
            _row("z", z, x.shape, dtype, dev, k) if z is not None else 0]
    if B.dim() not in (3, 4):
        raise ValueError("B and C are [B,T,N] or [B,T,G,N]")
    G = B.shape[2] if B.dim() == 4 else 1
    shape = (nb, T, G, N) if B.dim() == 4 else (nb, T, N)
    rows += [_row("B", B, shape, dtype, dev, len(shape) - 2), _row("C", C, shape, dtype, dev, len(shape) - 2)]
    _check_tokens(lengths, segments, nb, T, dev)
    fields = (nb, T, ch, N, G, _DT[dtype], _DT[y_dtype], _DT[grad_dtype], int(softplus), *rows)
    return fields, (nb,) + tok + (N,)


def lattice_osr_ssm_fwd(x, dt, A, B, C, state_in=None, *, D=None, z=None, dt_bias=None, softplus: bool = True,
                        lengths=None, segments=None, y_dtype=torch.float32, y=None, state_out=None, save: bool = False,
                        saved=None, workspace=None, stream=None):
    """h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t per channel and state, delta = softplus(dt + dt_bias) (or the
    sum itself), y_t = (sum_n C_t h_t + D x_t) z_t sigmoid(z_t) (no gate without z).

    x, dt, z [B,T,D] or [B,T,H,d] and B, C [B,T,N] or [B,T,G,N] (channel c takes group c // (D/G)) share a
    dtype, float32 or bfloat16; rows may be a stride of up to 2^22 elements apart, as in a slice of a projection's output.  A [D,N],
    D and dt_bias [D] are float32, state_in (None: zeros) and state_out [B,D,N] too, state_out may be
    state_in; lengths [B] int32: the tokens of each sequence, y is zero behind them; segments [B,T] int32: the
    document of every token, at whose borders the state starts from zero.
    Returns (y, state_out) and, with save (or `saved`, a uint8 tensor of lattice_osr_ssm_saved_bytes), what
    lattice_osr_ssm_bwd needs."""
    lib = load_library()
    fields, sshape = _ssm_desc(x, dt, A, B, C, D, z, dt_bias, softplus, lengths, segments, y_dtype, torch.float32)
    dev = x.device
    for name, t in (("state_in", state_in), ("state_out", state_out)):
        if t is not None:
            _check_tensor(name, t, sshape, torch.float32, dev)
    if y is not None:
        _check_tensor("y", y, x.shape, y_dtype, dev)
    _check_cuda(x)
    save = save or saved is not None

    def call(st):
        yy = x.new_empty(x.shape, dtype=y_dtype) if y is None else y
        so = x.new_empty(sshape, dtype=torch.float32) if state_out is None else state_out
        snb, wnb, _ = _ssm_sizes(fields)
        sv, sbytes = _room(saved, snb, x) if save else (None, 0)
        ws, wbytes = _room(workspace, wnb, x)
        rc = lib.lattice_osr_ssm_fwd(_ref(lattice_osr_ssm_desc, fields), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                                     _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(lengths), _ptr(segments), _ptr(state_in),
                                     _ptr(so), _ptr(yy), _ptr(sv), sbytes, _ptr(ws), wbytes, st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_ssm_fwd")
        return (yy, so, sv) if save else (yy, so)

    return _on(dev, stream, call)


def lattice_osr_ssm_bwd(x, dt, A, B, C, dy, dstate_out=None, *, saved, D=None, z=None, dt_bias=None,
                        softplus: bool = True, lengths=None, segments=None, grad_dtype=torch.float32,
                        grads: Optional[dict] = None, workspace=None, stream=None) -> dict:
    """Gradients of sum(dy*y) + sum(dstate_out*state_out) of lattice_osr_ssm_fwd with the same inputs, whose
    `saved` this call takes.  dy has x's shape (float32 or bfloat16), dstate_out the state's (None: zeros).
    Returns a dict of dx, ddt, dB, dC (and dz, with z) in grad_dtype, and dA, dstate_in (dD with D, ddt_bias
    with dt_bias) in float32, allocated unless passed in `grads`."""
    lib = load_library()
    if saved is None:
        raise ValueError("saved: the tensor lattice_osr_ssm_fwd returned with save=True")
    fields, sshape = _ssm_desc(x, dt, A, B, C, D, z, dt_bias, softplus, lengths, segments, dy.dtype, grad_dtype)
    dev = x.device
    _check_tensor("dy", dy, x.shape, None, dev)
    if dstate_out is not None:
        _check_tensor("dstate_out", dstate_out, sshape, torch.float32, dev)
    f32 = torch.float32
    want = [(n, None, t.shape, dt_) for n, t, dt_ in (("dx", x, grad_dtype), ("ddt", x, grad_dtype), ("dA", A, f32),
                                                     ("dB", B, grad_dtype), ("dC", C, grad_dtype), ("dD", D, f32),
                                                     ("dz", z, grad_dtype), ("ddt_bias", dt_bias, f32))
            if t is not None]
    want.append(("dstate_in", None, sshape, f32))
    _check_grads(grads, want, dev)
    _check_cuda(x)

    def call(st):
        g = _grads(grads, want, x)
        sv, sbytes = _workspace(saved, 0, dev)
        ws, wbytes = _room(workspace, _ssm_sizes(fields)[2], x)
        rc = lib.lattice_osr_ssm_bwd(_ref(lattice_osr_ssm_desc, fields), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                                     _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(lengths), _ptr(segments), _ptr(sv), sbytes,
                                     _ptr(dy), _ptr(dstate_out), _ptr(g["dx"]), _ptr(g["ddt"]), _ptr(g["dA"]),
                                     _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g.get("dD")), _ptr(g.get("dz")),
                                     _ptr(g.get("ddt_bias")), _ptr(g["dstate_in"]), _ptr(ws), wbytes, st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_ssm_bwd")
        return g

    return _on(dev, stream, call)


def lattice_osr_ssm_step(x, dt, A, B, C, state_in, *, D=None, z=None, dt_bias=None, softplus: bool = True,
                         y_dtype=torch.float32, y=None, state_out=None, stream=None):
    """One token of lattice_osr_ssm_fwd (T = 1) for every sequence; state_out may be state_in (in place).
    Returns (y, state_out)."""
    lib = load_library()
    if state_in is None:
        raise ValueError("state_in: the state of every sequence (zeros at its start)")
    fields, sshape = _ssm_desc(x, dt, A, B, C, D, z, dt_bias, softplus, None, None, y_dtype, torch.float32)
    dev = x.device
    _check_tensor("state_in", state_in, sshape, torch.float32, dev)
    if state_out is not None:
        _check_tensor("state_out", state_out, sshape, torch.float32, dev)
    if y is not None:
        _check_tensor("y", y, x.shape, y_dtype, dev)
    _check_cuda(x)

    def call(st):
        yy = x.new_empty(x.shape, dtype=y_dtype) if y is None else y
        so = torch.empty_like(state_in) if state_out is None else state_out
        rc = lib.lattice_osr_ssm_step(_ref(lattice_osr_ssm_desc, fields), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                                      _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(state_in), _ptr(so), _ptr(yy), st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_ssm_step")
        return yy, so

    return _on(dev, stream, call)


def make_layernorm_desc(R, D, in_dtype=BF16, res_dtype=BF16, grad_dtype=F32, eps=1e-5):
    return lattice_osr_layernorm_desc(R, D, in_dtype, res_dtype, grad_dtype, eps)


def lattice_osr_layernorm_bwd_workspace_bytes(desc: lattice_osr_layernorm_desc) -> int:
    return _bytes_of("lattice_osr_layernorm_bwd_workspace_bytes", desc)


@functools.lru_cache(maxsize=1024)
def _layernorm_size(fields):
    return _query("lattice_osr_layernorm_bwd_workspace_bytes", lattice_osr_layernorm_desc(*fields)) or 0


def _layernorm_desc(x, y, w, b, in_dtype, grad_dtype, eps):
    """Descriptor fields of a layer norm call, after checking every input against them."""
    if x.dim() < 1:
        raise ValueError("x and y are [..., D]")
    _check_dtypes(x.dtype, in_dtype, grad_dtype)
    dev, D = x.device, x.shape[-1]
    _check_tensor("x", x, x.shape, None)
    if y is not None:
        _check_tensor("y", y, x.shape, in_dtype, dev)
    for name, t in (("w", w), ("b", b)):
        if t is not None:
            _check_tensor(name, t, (D,), torch.float32, dev)
    R = x.numel() // D if D else 0
    if R > 2 ** 31 - 1:
        raise ValueError(f"{R} rows: at most 2^31 - 1")
    return R, D, _DT[in_dtype], _DT[x.dtype], _DT[grad_dtype], eps


def lattice_osr_layernorm_fwd(x, y=None, *, w=None, b=None, eps: float = 1e-5, z_dtype=None, x_out=None, z=None,
                              stream=None):
    """x_out = x + y (y None: x itself), z = (x_out - mean) / sqrt(var + eps) w + b over the last dimension.

    x [..., D] and y [..., D] have their own dtypes (float32 or bfloat16), z has y's (without y z_dtype, or
    x's if that is None); w, b are [D] float32 (None: ones, zeros).  x_out has x's dtype and may be x (in place).
    Returns (x_out, z); x_out is None without y."""
    lib = load_library()
    in_dtype = y.dtype if y is not None else z_dtype or x.dtype
    if z_dtype is not None and z_dtype != in_dtype:
        raise ValueError("z_dtype is y's dtype")
    fields = _layernorm_desc(x, y, w, b, in_dtype, torch.float32, eps)
    dev = x.device
    if x_out is not None:
        _check_tensor("x_out", x_out, x.shape, x.dtype, dev)
    if z is not None:
        _check_tensor("z", z, x.shape, in_dtype, dev)
    _check_cuda(x)

    def call(st):
        xo = torch.empty_like(x) if x_out is None and y is not None else x_out
        zz = torch.empty_like(x, dtype=in_dtype) if z is None else z
        rc = lib.lattice_osr_layernorm_fwd(_ref(lattice_osr_layernorm_desc, fields), _ptr(x), _ptr(y), _ptr(w),
                                           _ptr(b), _ptr(xo), _ptr(zz), st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_layernorm_fwd")
        return xo, zz

    return _on(dev, stream, call)


def lattice_osr_layernorm_bwd(x, y=None, dx_out=None, dz=None, *, w=None, b=None, eps: float = 1e-5, grad_dtype=None,
                              grads: Optional[dict] = None, workspace=None, stream=None) -> dict:
    """Gradients of sum(dx_out*x_out) + sum(dz*z) of lattice_osr_layernorm_fwd with the same inputs.  dx_out (x's
    dtype; None: zeros) and dz (y's dtype) have x's shape.  Returns a dict of dx (x's dtype), dy with y (grad_dtype,
    y's dtype if that is None; dx itself where that is x's dtype), dw and db (float32, where w and b were passed),
    allocated unless passed in `grads` (dx may be dx_out)."""
    lib = load_library()
    if dz is None:
        raise ValueError("dz: the gradient of z")
    in_dtype = y.dtype if y is not None else dz.dtype
    grad_dtype = in_dtype if grad_dtype is None else grad_dtype
    fields = _layernorm_desc(x, y, w, b, in_dtype, grad_dtype, eps)
    dev = x.device
    for name, t, dt in (("dx_out", dx_out, x.dtype), ("dz", dz, in_dtype)):
        if t is not None:
            _check_tensor(name, t, x.shape, dt, dev)
    f32 = torch.float32
    own_dy = y is not None and grad_dtype != x.dtype
    want = [(n, t, t.shape, dt) for n, t, dt in (("dx", x, x.dtype), ("dy", y if own_dy else None, grad_dtype),
                                                 ("dw", w, f32), ("db", b, f32)) if t is not None]
    _check_grads(grads, want, dev)
    _check_cuda(x)

    def call(st):
        g = _grads(grads, want, x)
        sums = w is not None or b is not None
        ws, wbytes = _room(workspace, _layernorm_size(fields) if sums else 0, x)
        rc = lib.lattice_osr_layernorm_bwd(_ref(lattice_osr_layernorm_desc, fields), _ptr(x), _ptr(y), _ptr(w),
                                           _ptr(dx_out), _ptr(dz), _ptr(g["dx"]), _ptr(g.get("dy")), _ptr(g.get("dw")),
                                           _ptr(g.get("db")), _ptr(ws), wbytes, st)
        if rc != OK:
            raise OSRError(rc, "lattice_osr_layernorm_bwd")
        if y is not None and not own_dy:
            g["dy"] = g["dx"]
        return g

    return _on(dev, stream, call)


def to_device(inp, device="cuda") -> dict:
    """Move an OSRInputs batch (numpy, storage form) to device tensors.

    bf16 bit patterns become torch.bfloat16 tensors with the same bits.
    """
    out = {}
    for name in ("q", "k", "v", "gamma", "mu"):
        a = getattr(inp, name)
        t = torch.from_numpy(a.copy())
        if a.dtype.itemsize == 2:
            t = t.view(torch.bfloat16)
        out[name] = t.to(device)
    out["state"] = torch.from_numpy(inp.state.copy()).to(device)
    return out
