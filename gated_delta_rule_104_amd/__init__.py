"""Python binding of libkda (Kimi Delta Attention on MI355X).

Argument marshalling only: every call checks tensor shapes, dtypes and devices,
allocates outputs with torch, and passes raw device pointers plus the current
HIP stream to the C-ABI in ``libkda.so`` (declared in ``include/libkda.h``).
All arithmetic runs in the library's HIP kernels; there is no fallback.  If the
library is missing, loading fails with an error that says how to build it.

Entry points (same names as the C-ABI):
    prefill(q, k, v, log_alpha, beta, S0=None)        -> (o, S_T)
    prefill_noalloc(q, k, v, log_alpha, beta, S0=None)  -> (o, S_T)  (no workspace, allocates nothing)
    prefill_snap(q, k, v, log_alpha, beta, snap_interval, S0=None) -> (o, S_T, S_snap)
    prefill_plan(B, H, T, dk, dv, dtype)               -> (T0, G, Tseg)
    prefill_segments(q, k, v, log_alpha, beta, S_start, Tseg) -> (o, S_T)
    decode_step(q, k, v, log_alpha, beta, S)           -> o          (S updated in place)
    decode_tokens(q, k, v, log_alpha, beta, S, S_out=None, positions=False) -> (o, S_pos or None)
    segment_transfer(k, v, log_alpha, beta, G)         -> (S_zero_end, M)
    segment_merge(S_zero_end, M, S_in=None)            -> (S_start, S_T)
    prefill_backward(q, k, v, log_alpha, beta, S0, dO, dS_T) -> dict of gradients
    conv_prefill(x, weight, bias=None, state=None, ...) -> (o, state_out)
    conv_step(x, state, weight, bias=None, ...)        -> o          (state moved on in place)
    conv_backward(x, weight, bias, state, dO, dstate_out=None, ...) -> dict of gradients
    ssm_prefill(q, k, v, log_alpha, beta, D=None, S0=None, ...) -> (o, S_T)
    ssm_step(q, k, v, log_alpha, beta, S, D=None)      -> o          (S updated in place)
    ssm_backward(q, k, v, log_alpha, beta, D, S0, dO, dS_T) -> dict of gradients
    state_cache(nslots, H, dk, dv, fmt, device)        -> (cache, scales)
    state_store(S, slots, cache, scales), state_load(cache, scales, slots) -> S
    set_option(name, value), get_option(name), options(**values) (context manager)
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Tuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkda.so")

KDA_F32, KDA_BF16 = 0, 1
_DT = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}
# status codes (include/libkda.h)
(KDA_OK, KDA_ERR_NULL, KDA_ERR_SHAPE, KDA_ERR_UNSUPPORTED, KDA_ERR_ALIGN, KDA_ERR_WORKSPACE,
 KDA_ERR_PRECONDITION, KDA_ERR_HIP) = range(8)

# kda_activation, kda_cache_format
_ACT = {None: 0, "silu": 1}
_CACHE = {torch.int8: 0, torch.float8_e4m3fn: 1}

_lib = None


class _Strides(ctypes.Structure):
    """kda_strides: elements between consecutive b, h, t."""
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("t", ctypes.c_longlong)]


class _SsmStrides(ctypes.Structure):
    """kda_ssm_strides."""
    _fields_ = [(n, _Strides) for n in ("q", "k", "v", "log_alpha", "beta", "o")]


class _SsmGradStrides(ctypes.Structure):
    """kda_ssm_grad_strides."""
    _fields_ = [(n, _Strides) for n in ("dO", "dq", "dk", "dv", "dlog_alpha", "dbeta")]


class KdaError(RuntimeError):
    """A libkda call returned a status other than KDA_OK (``status`` holds it;
    None for errors the binding itself raises)."""

    def __init__(self, msg: str, status: Optional[int] = None):
        super().__init__(msg)
        self.status = status


def lib_path() -> str:
    return LIB_PATH


def load() -> ctypes.CDLL:
    """Load libkda.so (built by ``python __graft_entry__.py`` / ``build.py``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise KdaError(f"libkda.so not found at {LIB_PATH}; build it with "
                       "`python gated_delta_rule_104_amd/build.py` (hipcc, gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i = ctypes.c_void_p, ctypes.c_int
    lib.kda_chunk_prefill.argtypes = [vp] * 8 + [i] * 6 + [vp, ctypes.c_size_t, vp]
    lib.kda_chunk_prefill_snap.argtypes = [vp] * 9 + [i] * 7 + [vp, ctypes.c_size_t, vp]
    lib.kda_chunk_prefill_noalloc.argtypes = [vp] * 8 + [i] * 6 + [vp]
    lib.kda_prefill_workspace_bytes.argtypes = [i] * 6
    lib.kda_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_prefill_plan.argtypes = [i] * 6 + [ctypes.POINTER(i)] * 3
    lib.kda_chunk_prefill_segments.argtypes = [vp] * 8 + [i] * 7 + [vp]
    lib.kda_decode_step.argtypes = [vp] * 7 + [i] * 5 + [vp]
    lib.kda_decode_tokens.argtypes = [vp] * 9 + [i] * 6 + [vp]
    lib.kda_segment_transfer.argtypes = [vp] * 6 + [i] * 7 + [vp]
    lib.kda_segment_merge.argtypes = [vp] * 5 + [i] * 5 + [vp]
    lib.kda_backward_workspace_bytes.argtypes = [i] * 6
    lib.kda_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_prefill_backward.argtypes = [vp] * 14 + [i] * 6 + [vp, ctypes.c_size_t, vp]
    sz, st = ctypes.c_size_t, ctypes.POINTER(_Strides)
    lib.kda_conv_prefill.argtypes = [vp, st, vp, vp, vp, vp, vp, st, vp] + [i] * 7 + [vp]
    lib.kda_conv_step.argtypes = [vp, st, vp, vp, vp, vp, st] + [i] * 6 + [vp]
    lib.kda_conv_backward_workspace_bytes.argtypes = [i] * 6
    lib.kda_conv_backward_workspace_bytes.restype = sz
    lib.kda_conv_backward.argtypes = [vp, st, vp, vp, vp, vp, st, vp, vp, st, vp, vp, vp] + [i] * 7 + [vp, sz, vp]
    lib.kda_ssm_prefill_workspace_bytes.argtypes = [i] * 7
    lib.kda_ssm_prefill_workspace_bytes.restype = sz
    lib.kda_ssm_prefill.argtypes = [vp] * 10 + [ctypes.POINTER(_SsmStrides)] + [i] * 7 + [vp, sz, vp]
    lib.kda_ssm_step.argtypes = [vp] * 8 + [i] * 6 + [vp]
    lib.kda_ssm_backward_workspace_bytes.argtypes = [i] * 7
    lib.kda_ssm_backward_workspace_bytes.restype = sz
    lib.kda_ssm_backward.argtypes = ([vp] * 16 + [ctypes.POINTER(_SsmStrides), ctypes.POINTER(_SsmGradStrides)] +
                                     [i] * 7 + [vp, sz, vp])
    lib.kda_state_store.argtypes = [vp] * 4 + [i] * 6 + [vp]
    lib.kda_state_load.argtypes = [vp] * 4 + [i] * 6 + [vp]
    for f in (lib.kda_conv_prefill, lib.kda_conv_step, lib.kda_conv_backward, lib.kda_ssm_prefill, lib.kda_ssm_step,
              lib.kda_ssm_backward, lib.kda_state_store, lib.kda_state_load):
        f.restype = i
    for f in (lib.kda_chunk_prefill, lib.kda_chunk_prefill_snap, lib.kda_chunk_prefill_noalloc, lib.kda_prefill_plan, lib.kda_chunk_prefill_segments,
              lib.kda_decode_step, lib.kda_decode_tokens, lib.kda_segment_transfer,
              lib.kda_segment_merge, lib.kda_prefill_backward):
        f.restype = i
    lib.kda_set_option.argtypes = [ctypes.c_char_p, ctypes.c_longlong]
    lib.kda_set_option.restype = i
    lib.kda_get_option.argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_longlong)]
    lib.kda_get_option.restype = i
    lib.kda_status_string.argtypes = [i]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_last_error.restype = ctypes.c_char_p
    lib.kda_abi_version.restype = i
    lib.kda_debug_time_main_launches.argtypes = [i]
    lib.kda_debug_time_main_launches.restype = i
    lib.kda_debug_main_launch_ms.argtypes = [ctypes.POINTER(ctypes.c_float), i, ctypes.POINTER(i)]
    lib.kda_debug_main_launch_ms.restype = i
    _lib = lib
    return lib


def _check(rc: int, what: str) -> None:
    if rc != 0:
        lib = load()
        raise KdaError(f"{what}: {lib.kda_status_string(rc).decode()} "
                       f"({lib.kda_last_error().decode()})", rc)


def set_option(name: str, value: Optional[int]) -> None:
    """Set a process-wide library option (kda_set_option); None restores the default."""
    _check(load().kda_set_option(name.encode(), -1 if value is None else int(value)), f"set_option({name})")


def get_option(name: str) -> Optional[int]:
    """The option's value in effect, or None for the library's default."""
    v = ctypes.c_longlong(0)
    _check(load().kda_get_option(name.encode(), ctypes.byref(v)), f"get_option({name})")
    return None if v.value == -1 else int(v.value)


def debug_time_main_launches(count: int) -> None:
    """Arm HIP events around the main launch of the next `count` sequence-split
    prefills (kda_debug_time_main_launches; 0 disarms)."""
    _check(load().kda_debug_time_main_launches(int(count)), "debug_time_main_launches")


def debug_main_launch_ms() -> list:
    """Durations (ms) of the main launches timed since the arming
    (kda_debug_main_launch_ms; waits for them)."""
    lib = load()
    n = ctypes.c_int(0)
    _check(lib.kda_debug_main_launch_ms(None, 0, ctypes.byref(n)), "debug_main_launch_ms")
    buf = (ctypes.c_float * max(n.value, 1))()
    _check(lib.kda_debug_main_launch_ms(buf, n.value, ctypes.byref(n)), "debug_main_launch_ms")
    return [float(buf[i]) for i in range(n.value)]


@contextlib.contextmanager
def options(**values):
    """Set options for the duration of a with-block, then restore the old values."""
    old = {n: get_option(n) for n in values}
    try:
        for n, v in values.items():
            set_option(n, v)
        yield
    finally:
        for n, v in old.items():
            set_option(n, v)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# (the same handle as current_stream().cuda_stream, without building a Stream: 0.1 us, not 2.5)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream() -> int:
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _io(t: torch.Tensor, name: str, dtype: torch.dtype, shape) -> None:
    if not t.is_cuda:
        raise KdaError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise KdaError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise KdaError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise KdaError(f"{name} must be contiguous")


def prefill_workspace_bytes(B: int, H: int, T: int, dk: int, dv: int, dtype: torch.dtype) -> int:
    """Workspace that lets kda_chunk_prefill use its sequence-split path (0 if unused)."""
    if dtype not in _DT:
        raise KdaError(f"unsupported dtype {dtype}")
    return int(load().kda_prefill_workspace_bytes(B, H, T, dk, dv, _DT[dtype]))


def prefill(q, k, v, log_alpha, beta, S0=None, o=None, S_T=None,
            workspace="auto") -> Tuple[torch.Tensor, torch.Tensor]:
    """Chunked prefill.  q, k, log_alpha [B,H,T,dk]; v [B,H,T,dv]; beta [B,H,T];
    S0 [B,H,dk,dv] fp32 or None.  Returns o [B,H,T,dv] (input dtype) and S_T fp32.
    workspace: "auto" allocates what kda_prefill_workspace_bytes asks for, None
    passes none (single-pass path), or a device uint8 tensor to use."""
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    dt = k.dtype
    if dt not in _DT:
        raise KdaError(f"unsupported dtype {dt}")
    for name, t, shp in (("q", q, (B, H, T, dk)), ("k", k, (B, H, T, dk)), ("v", v, (B, H, T, dv)),
                         ("log_alpha", log_alpha, (B, H, T, dk)), ("beta", beta, (B, H, T))):
        _io(t, name, dt, shp)
    if S0 is not None:
        _io(S0, "S0", torch.float32, (B, H, dk, dv))
    if o is None:
        o = torch.empty(B, H, T, dv, dtype=dt, device=k.device)
    if S_T is None:
        S_T = torch.empty(B, H, dk, dv, dtype=torch.float32, device=k.device)
    _io(o, "o", dt, (B, H, T, dv))
    _io(S_T, "S_T", torch.float32, (B, H, dk, dv))
    if isinstance(workspace, str):
        nbytes = prefill_workspace_bytes(B, H, T, dk, dv, dt)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=k.device) if nbytes else None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().kda_chunk_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0),
                                  _ptr(o), _ptr(S_T), B, H, T, dk, dv, _DT[dt], _ptr(workspace),
                                  ws_bytes, _stream())
    _check(rc, "kda_chunk_prefill")
    return o, S_T


def prefill_noalloc(q, k, v, log_alpha, beta, S0=None, o=None, S_T=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """prefill() through kda_chunk_prefill_noalloc: the library's own scratch
    array replaces the workspace (calls on one device must not overlap).  o and
    S_T are allocated here when not given; pass them to allocate nothing."""
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    dt = k.dtype
    if dt not in _DT:
        raise KdaError(f"unsupported dtype {dt}")
    for name, t, shp in (("q", q, (B, H, T, dk)), ("k", k, (B, H, T, dk)), ("v", v, (B, H, T, dv)),
                         ("log_alpha", log_alpha, (B, H, T, dk)), ("beta", beta, (B, H, T))):
        _io(t, name, dt, shp)
    if S0 is not None:
        _io(S0, "S0", torch.float32, (B, H, dk, dv))
    if o is None:
        o = torch.empty(B, H, T, dv, dtype=dt, device=k.device)
    if S_T is None:
        S_T = torch.empty(B, H, dk, dv, dtype=torch.float32, device=k.device)
    _io(o, "o", dt, (B, H, T, dv))
    _io(S_T, "S_T", torch.float32, (B, H, dk, dv))
    rc = load().kda_chunk_prefill_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0),
                                          _ptr(o), _ptr(S_T), B, H, T, dk, dv, _DT[dt], _stream())
    _check(rc, "kda_chunk_prefill_noalloc")
    return o, S_T


def prefill_snap(q, k, v, log_alpha, beta, snap_interval: int, S0=None, o=None, S_T=None,
                 S_snap=None, workspace="auto"):
    """Chunked prefill that also returns state snapshots for prefix caching:
    S_snap [B, T // snap_interval, H, dk, dv] fp32, entry [b, j, h] being the state
    after the first (j + 1) * snap_interval tokens (snap_interval: a positive
    multiple of 64).  Returns (o, S_T, S_snap); o and S_T are those of prefill()."""
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    dt = k.dtype
    if dt not in _DT:
        raise KdaError(f"unsupported dtype {dt}")
    if snap_interval <= 0 or snap_interval % 64:
        raise KdaError(f"snap_interval must be a positive multiple of 64 (got {snap_interval})")
    for name, t, shp in (("q", q, (B, H, T, dk)), ("k", k, (B, H, T, dk)), ("v", v, (B, H, T, dv)),
                         ("log_alpha", log_alpha, (B, H, T, dk)), ("beta", beta, (B, H, T))):
        _io(t, name, dt, shp)
    if S0 is not None:
        _io(S0, "S0", torch.float32, (B, H, dk, dv))
    nsnap = T // snap_interval
    if o is None:
        o = torch.empty(B, H, T, dv, dtype=dt, device=k.device)
    if S_T is None:
        S_T = torch.empty(B, H, dk, dv, dtype=torch.float32, device=k.device)
    if S_snap is None:
        S_snap = torch.empty(B, nsnap, H, dk, dv, dtype=torch.float32, device=k.device)
    _io(o, "o", dt, (B, H, T, dv))
    _io(S_T, "S_T", torch.float32, (B, H, dk, dv))
    _io(S_snap, "S_snap", torch.float32, (B, nsnap, H, dk, dv))
    if isinstance(workspace, str):
        nbytes = prefill_workspace_bytes(B, H, T, dk, dv, dt)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=k.device) if nbytes else None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().kda_chunk_prefill_snap(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                       _ptr(S0), _ptr(o), _ptr(S_T), _ptr(S_snap) if nsnap else None,
                                       snap_interval, B, H, T, dk, dv, _DT[dt], _ptr(workspace),
                                       ws_bytes, _stream())
    _check(rc, "kda_chunk_prefill_snap")
    return o, S_T, S_snap


def prefill_plan(B: int, H: int, T: int, dk: int, dv: int, dtype: torch.dtype) -> Tuple[int, int, int]:
    """(T0, G, Tseg): the cut kda_chunk_prefill uses with its workspace: a first
    part of T0 tokens, then G segments of Tseg tokens (T0 == 0, G == 1: single pass)."""
    if dtype not in _DT:
        raise KdaError(f"unsupported dtype {dtype}")
    T0, G, Tseg = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(load().kda_prefill_plan(B, H, T, dk, dv, _DT[dtype], ctypes.byref(T0), ctypes.byref(G),
                                   ctypes.byref(Tseg)), "kda_prefill_plan")
    return T0.value, G.value, Tseg.value


def prefill_segments(q, k, v, log_alpha, beta, S_start, Tseg: int, o=None, S_T=None):
    """Prefill of the G = ceil(T / Tseg) segments of every head, segment i from
    S_start[i] ([G,B,H,dk,dv] fp32, or None for zero).  Returns (o, S_T of the
    last segment)."""
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    dt = k.dtype
    if dt not in _DT:
        raise KdaError(f"unsupported dtype {dt}")
    if Tseg < 1 or T < 1:
        raise KdaError(f"need T >= 1 and Tseg >= 1 (T={T}, Tseg={Tseg})")
    G = -(-T // Tseg)
    for name, t, shp in (("q", q, (B, H, T, dk)), ("k", k, (B, H, T, dk)), ("v", v, (B, H, T, dv)),
                         ("log_alpha", log_alpha, (B, H, T, dk)), ("beta", beta, (B, H, T))):
        _io(t, name, dt, shp)
    if S_start is not None:
        _io(S_start, "S_start", torch.float32, (G, B, H, dk, dv))
    if o is None:
        o = torch.empty(B, H, T, dv, dtype=dt, device=k.device)
    if S_T is None:
        S_T = torch.empty(B, H, dk, dv, dtype=torch.float32, device=k.device)
    _io(o, "o", dt, (B, H, T, dv))
    _io(S_T, "S_T", torch.float32, (B, H, dk, dv))
    rc = load().kda_chunk_prefill_segments(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                           _ptr(S_start), _ptr(o), _ptr(S_T), B, H, T, Tseg, dk, dv,
                                           _DT[dt], _stream())
    _check(rc, "kda_chunk_prefill_segments")
    return o, S_T


def decode_step(q, k, v, log_alpha, beta, S, o=None) -> torch.Tensor:
    """One token for N*H heads.  q, k, log_alpha [N,H,dk]; v [N,H,dv]; beta [N,H];
    S [N,H,dk,dv] fp32, updated in place.  Returns o [N,H,dv]."""
    N, H, dk = k.shape
    dv = v.shape[-1]
    dt = k.dtype
    if dt not in _DT:
        raise KdaError(f"unsupported dtype {dt}")
    for name, t, shp in (("q", q, (N, H, dk)), ("k", k, (N, H, dk)), ("v", v, (N, H, dv)),
                         ("log_alpha", log_alpha, (N, H, dk)), ("beta", beta, (N, H))):
        _io(t, name, dt, shp)
    _io(S, "S", torch.float32, (N, H, dk, dv))
    if o is None:
        o = torch.empty(N, H, dv, dtype=dt, device=k.device)
    _io(o, "o", dt, (N, H, dv))
    rc = load().kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S),
                                _ptr(o), N, H, dk, dv, _DT[dt], _stream())
    _check(rc, "kda_decode_step")
    return o


def decode_tokens(q, k, v, log_alpha, beta, S, S_out=None, positions: bool = False, o=None, S_pos=None):
    """ntok consecutive tokens per sequence in one pass over the state (speculative
    decoding's verification step).  q, k, log_alpha [N,H,ntok,dk]; v [N,H,ntok,dv];
    beta [N,H,ntok]; S [N,H,dk,dv] fp32.  The state after the tokens goes to S_out
    (default: S itself, in place).  With positions=True (or an S_pos tensor) the
    state after each token is returned too, [N,ntok,H,dk,dv].  Returns (o, S_pos)."""
    N, H, ntok, dk = k.shape
    dv = v.shape[-1]
    dt = k.dtype
    if dt not in _DT:
        raise KdaError(f"unsupported dtype {dt}")
    for name, t, shp in (("q", q, (N, H, ntok, dk)), ("k", k, (N, H, ntok, dk)), ("v", v, (N, H, ntok, dv)),
                         ("log_alpha", log_alpha, (N, H, ntok, dk)), ("beta", beta, (N, H, ntok))):
        _io(t, name, dt, shp)
    _io(S, "S", torch.float32, (N, H, dk, dv))
    if S_out is None:
        S_out = S
    _io(S_out, "S_out", torch.float32, (N, H, dk, dv))
    if o is None:
        o = torch.empty(N, H, ntok, dv, dtype=dt, device=k.device)
    _io(o, "o", dt, (N, H, ntok, dv))
    if S_pos is None and positions:
        S_pos = torch.empty(N, ntok, H, dk, dv, dtype=torch.float32, device=k.device)
    if S_pos is not None:
        _io(S_pos, "S_pos", torch.float32, (N, ntok, H, dk, dv))
    rc = load().kda_decode_tokens(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S),
                                  _ptr(S_out), _ptr(o), _ptr(S_pos), N, H, ntok, dk, dv, _DT[dt], _stream())
    _check(rc, "kda_decode_tokens")
    return o, S_pos


def segment_transfer(k, v, log_alpha, beta, G: int, S_zero_end=None, M=None):
    """Per-segment zero-start end states [G,B,H,dk,dv] and transfer maps [G,B,H,dk,dk]
    for sequences of T = G * Tseg tokens."""
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    dt = k.dtype
    if dt not in _DT:
        raise KdaError(f"unsupported dtype {dt}")
    if G <= 0 or T % G:
        raise KdaError(f"T={T} is not a positive multiple of G={G}")
    for name, t, shp in (("k", k, (B, H, T, dk)), ("v", v, (B, H, T, dv)),
                         ("log_alpha", log_alpha, (B, H, T, dk)), ("beta", beta, (B, H, T))):
        _io(t, name, dt, shp)
    if S_zero_end is None:
        S_zero_end = torch.empty(G, B, H, dk, dv, dtype=torch.float32, device=k.device)
    if M is None:
        M = torch.empty(G, B, H, dk, dk, dtype=torch.float32, device=k.device)
    _io(S_zero_end, "S_zero_end", torch.float32, (G, B, H, dk, dv))
    _io(M, "M", torch.float32, (G, B, H, dk, dk))
    rc = load().kda_segment_transfer(_ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S_zero_end),
                                     _ptr(M), B, H, G, T // G, dk, dv, _DT[dt], _stream())
    _check(rc, "kda_segment_transfer")
    return S_zero_end, M


def segment_merge(S_zero_end, M, S_in=None, want_start: bool = True, S_start=None, S_T=None):
    """Sequential merge.  Returns (S_start [G,B,H,dk,dv] or None, S_T [B,H,dk,dv])."""
    G, B, H, dk, dv = S_zero_end.shape
    _io(S_zero_end, "S_zero_end", torch.float32, (G, B, H, dk, dv))
    _io(M, "M", torch.float32, (G, B, H, dk, dk))
    if S_in is not None:
        _io(S_in, "S_in", torch.float32, (B, H, dk, dv))
    if want_start and S_start is None:
        S_start = torch.empty_like(S_zero_end)
    if S_start is not None:
        _io(S_start, "S_start", torch.float32, (G, B, H, dk, dv))
    if S_T is None:
        S_T = torch.empty(B, H, dk, dv, dtype=torch.float32, device=M.device)
    _io(S_T, "S_T", torch.float32, (B, H, dk, dv))
    rc = load().kda_segment_merge(_ptr(S_in), _ptr(S_zero_end), _ptr(M), _ptr(S_start), _ptr(S_T),
                                  B, H, G, dk, dv, _stream())
    _check(rc, "kda_segment_merge")
    return S_start, S_T


def backward_workspace_bytes(B: int, H: int, T: int, dk: int, dv: int, dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace kda_prefill_backward needs for inputs of this dtype (0 for an unsupported shape)."""
    if dtype not in _DT:
        raise KdaError(f"unsupported dtype {dtype}")
    return int(load().kda_backward_workspace_bytes(B, H, T, dk, dv, _DT[dtype]))


def prefill_backward(q, k, v, log_alpha, beta, S0=None, dO=None, dS_T=None, workspace=None):
    """Gradients of L = sum(dO * o) + sum(dS_T * S_T) of the prefill with respect
    to its inputs.  Returns a dict: dq, dk, dlog_alpha [B,H,T,dk], dv [B,H,T,dv],
    dbeta [B,H,T] in the inputs' dtype, and dS0 [B,H,dk,dv] fp32."""
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    dt = k.dtype
    if dt not in _DT:
        raise KdaError(f"unsupported dtype {dt}")
    for t, n, shp in ((q, "q", (B, H, T, dk)), (k, "k", (B, H, T, dk)), (v, "v", (B, H, T, dv)),
                      (log_alpha, "log_alpha", (B, H, T, dk)), (beta, "beta", (B, H, T))):
        _io(t, n, dt, shp)
    if S0 is not None:
        _io(S0, "S0", torch.float32, (B, H, dk, dv))
    if dO is not None:
        _io(dO, "dO", dt, (B, H, T, dv))
    if dS_T is not None:
        _io(dS_T, "dS_T", torch.float32, (B, H, dk, dv))
    dev = k.device
    io = dict(dtype=dt, device=dev)
    out = dict(dq=torch.empty(B, H, T, dk, **io), dk=torch.empty(B, H, T, dk, **io),
               dv=torch.empty(B, H, T, dv, **io), dlog_alpha=torch.empty(B, H, T, dk, **io),
               dbeta=torch.empty(B, H, T, **io), dS0=torch.empty(B, H, dk, dv, dtype=torch.float32, device=dev))
    need = backward_workspace_bytes(B, H, T, dk, dv, dt)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    if not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise KdaError(f"workspace must be a device tensor of at least {need} bytes")
    rc = load().kda_prefill_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0), _ptr(dO),
                                     _ptr(dS_T), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                                     _ptr(out["dlog_alpha"]), _ptr(out["dbeta"]), _ptr(out["dS0"]), B, H, T, dk, dv,
                                     _DT[dt], _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream())
    _check(rc, "kda_prefill_backward")
    return out


# ------------------------------------------------------- companion operators
# (These calls take microseconds: what is right is checked in one expression, and
# only what is wrong is looked at again to say why.)
def _device(t: torch.Tensor, name: str) -> torch.device:
    """The current device, on whose current stream the call runs; t has to be there."""
    if not t.is_cuda:
        raise KdaError(f"{name} must be a device tensor")
    if t.device.index != torch.cuda.current_device():
        raise KdaError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return t.device


def _wrong(t: torch.Tensor, name: str, dtype: torch.dtype, shape, dev: torch.device) -> None:
    if not t.is_cuda:
        raise KdaError(f"{name} must be a device tensor")
    if t.device != dev:
        raise KdaError(f"{name} is on {t.device}, expected {dev}")
    _io(t, name, dtype, shape)


def _dense(t: torch.Tensor, name: str, dtype: torch.dtype, shape, dev: torch.device) -> None:
    if t.device != dev or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        _wrong(t, name, dtype, shape, dev)


def _view(t: torch.Tensor, name: str, dtype: torch.dtype, shape, dev: torch.device, rows: bool = True) -> _Strides:
    """A [B, H, T] or (rows) [B, H, T, d] tensor with any strides but a contiguous last
    dimension of rows; the library checks their alignment."""
    st = t.stride()
    if t.device != dev or t.dtype != dtype or t.shape != shape:
        _wrong(t, name, dtype, shape, dev)
        raise KdaError(f"{name} does not fit")
    if rows and st[-1] != 1 and shape[-1] > 1:
        raise KdaError(f"{name} must have contiguous rows")
    return _Strides(*st[:3])


def _new_like(t: torch.Tensor, dtype=None) -> torch.Tensor:
    """A new tensor in the memory order of t where t is dense, contiguous otherwise."""
    return torch.empty_like(t, dtype=dtype or t.dtype)


def _scratch(workspace, need: int, device) -> torch.Tensor:
    if workspace is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    if workspace.device != device:
        raise KdaError(f"workspace is on {workspace.device}, expected {device}")
    if not workspace.is_contiguous() or workspace.numel() * workspace.element_size() < need:
        raise KdaError(f"workspace must be a contiguous device tensor of at least {need} bytes")
    return workspace


def _dtype(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise KdaError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def _rank(t: torch.Tensor, name: str, n: int) -> None:
    if t.dim() != n:
        raise KdaError(f"{name} has {t.dim()} dimensions, expected {n}")


def _act(activation) -> int:
    if activation not in _ACT:
        raise KdaError(f"unknown activation {activation!r} (None or 'silu')")
    return _ACT[activation]


def _conv_args(x, weight, bias, state, B, H, d, dev):
    _rank(weight, "weight", 3)
    K = weight.shape[2]
    _dense(weight, "weight", x.dtype, (H, d, K), dev)
    if bias is not None:
        _dense(bias, "bias", x.dtype, (H, d), dev)
    if state is not None:
        _dense(state, "state", x.dtype, (B, H, K - 1, d), dev)
    return K


def conv_prefill(x, weight, bias=None, state=None, activation="silu", lens=None, o=None, state_out=None):
    """Short causal convolution with K taps per channel (kda_conv_prefill).  x [B,H,T,d] (strides
    free, rows contiguous: a projection's [B,T,H*d] output as .view(B,T,H,d).transpose(1,2)),
    weight [H,d,K], bias [H,d], state [B,H,K-1,d] (the tokens before, or None), lens [B] int32 or
    None.  Returns o (contiguous unless given, rows behind lens not written) and the state after
    the sequence."""
    _rank(x, "x", 4)
    B, H, T, d = x.shape
    dt, dev = _dtype(x), _device(x, "x")
    xs = _view(x, "x", x.dtype, (B, H, T, d), dev)
    K = _conv_args(x, weight, bias, state, B, H, d, dev)
    if lens is not None:
        _dense(lens, "lens", torch.int32, (B,), dev)
    if o is None:
        o = torch.empty(B, H, T, d, dtype=x.dtype, device=x.device)
    os_ = _view(o, "o", x.dtype, (B, H, T, d), dev)
    if state_out is None:
        state_out = torch.empty(B, H, K - 1, d, dtype=x.dtype, device=x.device)
    _dense(state_out, "state_out", x.dtype, (B, H, K - 1, d), dev)
    rc = load().kda_conv_prefill(_ptr(x), xs, _ptr(weight), _ptr(bias), _ptr(state), _ptr(lens), _ptr(o), os_,
                                 _ptr(state_out), B, H, T, d, K, _act(activation), dt, _stream())
    _check(rc, "kda_conv_prefill")
    return o, state_out


def conv_step(x, state, weight, bias=None, activation="silu", o=None) -> torch.Tensor:
    """One token of the convolution: x [N,H,d] (strides free), state [N,H,K-1,d] moved on in
    place.  Returns o [N,H,d]."""
    _rank(x, "x", 3)
    N, H, d = x.shape
    dt, dev = _dtype(x), _device(x, "x")
    xs = _view(x, "x", x.dtype, (N, H, d), dev)
    K = _conv_args(x, weight, bias, state, N, H, d, dev)
    if state is None:
        raise KdaError("state is required")
    if o is None:
        o = torch.empty(N, H, d, dtype=x.dtype, device=x.device)
    os_ = _view(o, "o", x.dtype, (N, H, d), dev)
    rc = load().kda_conv_step(_ptr(x), xs, _ptr(state), _ptr(weight), _ptr(bias), _ptr(o), os_, N, H, d, K,
                              _act(activation), dt, _stream())
    _check(rc, "kda_conv_step")
    return o


def conv_backward(x, weight, bias, state, dO, dstate_out=None, activation="silu", workspace=None):
    """Gradients of conv_prefill (without lens).  Returns a dict: dx, dweight, and dbias and dstate
    where bias and state were given, in x's dtype."""
    _rank(x, "x", 4)
    B, H, T, d = x.shape
    dt, dev = _dtype(x), _device(x, "x")
    xs = _view(x, "x", x.dtype, (B, H, T, d), dev)
    K = _conv_args(x, weight, bias, state, B, H, d, dev)
    dos = _view(dO, "dO", x.dtype, (B, H, T, d), dev)
    if dstate_out is not None:
        _dense(dstate_out, "dstate_out", x.dtype, (B, H, K - 1, d), dev)
    out = dict(dx=_new_like(x), dweight=_new_like(weight))
    if bias is not None:
        out["dbias"] = _new_like(bias)
    if state is not None:
        out["dstate"] = _new_like(state)
    lib = load()
    need = int(lib.kda_conv_backward_workspace_bytes(B, H, T, d, K, dt))
    workspace = _scratch(workspace, need, x.device)
    rc = lib.kda_conv_backward(_ptr(x), xs, _ptr(weight), _ptr(bias), _ptr(state), _ptr(dO), dos, _ptr(dstate_out),
                               _ptr(out["dx"]), _Strides(*out["dx"].stride()[:3]), _ptr(out["dweight"]),
                               _ptr(out.get("dbias")), _ptr(out.get("dstate")), B, H, T, d, K, _act(activation), dt,
                               _ptr(workspace), workspace.numel() * workspace.element_size(), _stream())
    _check(rc, "kda_conv_backward")
    return out


def _ssm_args(q, k, v, log_alpha, beta, D, S0):
    _rank(k, "k", 4)
    _rank(v, "v", 4)
    (B, G, T, dk), (H, dv) = k.shape, (v.shape[1], v.shape[3])
    dt, dev = v.dtype, _device(v, "v")
    st = _SsmStrides(_view(q, "q", dt, (B, G, T, dk), dev), _view(k, "k", dt, (B, G, T, dk), dev),
                     _view(v, "v", dt, (B, H, T, dv), dev),
                     _view(log_alpha, "log_alpha", dt, (B, H, T), dev, rows=False),
                     _view(beta, "beta", dt, (B, H, T), dev, rows=False))
    if D is not None:
        _dense(D, "D", dt, (H,), dev)
    if S0 is not None:
        _dense(S0, "S0", torch.float32, (B, H, dk, dv), dev)
    return (B, H, G, T, dk, dv), st, dev


def ssm_prefill_workspace_bytes(B: int, H: int, G: int, T: int, dk: int, dv: int, dtype: torch.dtype) -> int:
    """Workspace with which kda_ssm_prefill may cut the sequences into segments (0: it would not)."""
    if dtype not in _DT:
        raise KdaError(f"unsupported dtype {dtype}")
    return int(load().kda_ssm_prefill_workspace_bytes(B, H, G, T, dk, dv, _DT[dtype]))


def ssm_prefill(q, k, v, log_alpha, beta, D=None, S0=None, lens=None, o=None, S_T=None, workspace="auto"):
    """Selective state space scan over a prompt (kda_ssm_prefill): per head
    S_t = exp(log_alpha_t) S_{t-1} + beta_t k_t v_t^T, o_t = S_t^T q_t + D v_t.  q, k [B,G,T,dk]
    shared by the H / G heads of a group, v [B,H,T,dv], log_alpha, beta [B,H,T] (strides free, rows
    contiguous), D [H] or None, S0 [B,H,dk,dv] fp32 or None, lens [B] int32 or None.  Returns o (in
    v's memory order unless given, rows behind lens not written) and S_T fp32.  workspace: "auto",
    None (each sequence in one piece) or a device uint8 tensor."""
    dt = _dtype(v)
    (B, H, G, T, dk, dv), st, dev = _ssm_args(q, k, v, log_alpha, beta, D, S0)
    if lens is not None:
        _dense(lens, "lens", torch.int32, (B,), dev)
    if o is None:
        o = _new_like(v)
    st.o = _view(o, "o", v.dtype, (B, H, T, dv), dev)
    if S_T is None:
        S_T = torch.empty(B, H, dk, dv, dtype=torch.float32, device=v.device)
    _dense(S_T, "S_T", torch.float32, (B, H, dk, dv), dev)
    lib = load()
    if isinstance(workspace, str):
        need = int(lib.kda_ssm_prefill_workspace_bytes(B, H, G, T, dk, dv, dt))
        workspace = torch.empty(need, dtype=torch.uint8, device=v.device) if need else None
    elif workspace is not None:
        _scratch(workspace, 0, v.device)
    rc = lib.kda_ssm_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(D), _ptr(S0), _ptr(lens),
                             _ptr(o), _ptr(S_T), st, B, H, G, T, dk, dv, dt, _ptr(workspace),
                             0 if workspace is None else workspace.numel() * workspace.element_size(), _stream())
    _check(rc, "kda_ssm_prefill")
    return o, S_T


def ssm_step(q, k, v, log_alpha, beta, S, D=None, o=None) -> torch.Tensor:
    """One token of the scan: q, k [N,G,dk], v [N,H,dv], log_alpha, beta [N,H], S [N,H,dk,dv] fp32
    updated in place.  Returns o [N,H,dv]."""
    _rank(k, "k", 3)
    _rank(v, "v", 3)
    (N, G, dk), (H, dv) = k.shape, v.shape[1:]
    dt, dev = _dtype(v), _device(v, "v")
    for name, t, shp in (("q", q, (N, G, dk)), ("k", k, (N, G, dk)), ("v", v, (N, H, dv)),
                         ("log_alpha", log_alpha, (N, H)), ("beta", beta, (N, H))):
        _dense(t, name, v.dtype, shp, dev)
    if D is not None:
        _dense(D, "D", v.dtype, (H,), dev)
    _dense(S, "S", torch.float32, (N, H, dk, dv), dev)
    if o is None:
        o = torch.empty(N, H, dv, dtype=v.dtype, device=dev)
    else:
        _dense(o, "o", v.dtype, (N, H, dv), dev)
    rc = load().kda_ssm_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(D), _ptr(S), _ptr(o),
                             N, H, G, dk, dv, dt, _stream())
    _check(rc, "kda_ssm_step")
    return o


def ssm_backward(q, k, v, log_alpha, beta, D=None, S0=None, dO=None, dS_T=None, workspace=None):
    """Gradients of L = sum(dO * o) + sum(dS_T * S_T) of ssm_prefill (without lens).  Returns a dict:
    dq, dk (summed over a group's heads), dv, dlog_alpha, dbeta, and dD and dS0 (fp32) where D and S0
    were given."""
    dt = _dtype(v)
    (B, H, G, T, dk, dv), st, dev = _ssm_args(q, k, v, log_alpha, beta, D, S0)
    if dO is None:
        raise KdaError("dO is required")
    if dS_T is not None:
        _dense(dS_T, "dS_T", torch.float32, (B, H, dk, dv), dev)
    out = dict(dq=_new_like(q), dk=_new_like(k), dv=_new_like(v), dlog_alpha=_new_like(log_alpha), dbeta=_new_like(beta))
    gst = _SsmGradStrides(dO=_view(dO, "dO", v.dtype, (B, H, T, dv), dev),
                          **{n: _Strides(*t.stride()[:3]) for n, t in out.items()})
    if D is not None:
        out["dD"] = _new_like(D)
    if S0 is not None:
        out["dS0"] = _new_like(S0)
    lib = load()
    need = int(lib.kda_ssm_backward_workspace_bytes(B, H, G, T, dk, dv, dt))
    workspace = _scratch(workspace, need, v.device)
    rc = lib.kda_ssm_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(D), _ptr(S0), _ptr(dO),
                              _ptr(dS_T), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dlog_alpha"]),
                              _ptr(out["dbeta"]), _ptr(out.get("dD")), _ptr(out.get("dS0")), st, gst, B, H, G, T, dk, dv,
                              dt, _ptr(workspace), workspace.numel() * workspace.element_size(), _stream())
    _check(rc, "kda_ssm_backward")
    return out


def state_cache(nslots: int, H: int, dk: int, dv: int, fmt: str = "int8", device="cuda"):
    """An empty quantised state cache: values [nslots,H,dk,dv] ("int8", or "e4m3" as
    torch.float8_e4m3fn) and scale exponents [nslots,H,dk,dv/32] uint8."""
    if fmt not in ("int8", "e4m3"):
        raise KdaError(f"unknown cache format {fmt!r} ('int8' or 'e4m3')")
    if dv % 32:
        raise KdaError(f"rows of {dv} values are not whole blocks of 32")
    cache = torch.zeros(nslots, H, dk, dv, dtype=torch.uint8, device=device)
    return (cache.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn),
            torch.ones(nslots, H, dk, dv // 32, dtype=torch.uint8, device=device))


def _cache_args(cache, scales, slots):
    _rank(cache, "cache", 4)
    if cache.dtype not in _CACHE:
        raise KdaError(f"cache has dtype {cache.dtype}, expected torch.int8 or torch.float8_e4m3fn")
    nslots, H, dk, dv = cache.shape
    dev = _device(cache, "cache")
    _dense(cache, "cache", cache.dtype, cache.shape, dev)
    _dense(scales, "scales", torch.uint8, (nslots, H, dk, dv // 32), dev)
    _rank(slots, "slots", 1)
    _dense(slots, "slots", torch.int32, slots.shape, dev)
    return nslots, H, dk, dv, dev


def state_store(S, slots, cache, scales) -> None:
    """Quantise states S [..., H,dk,dv] fp32 into the entries slots [n] int32 of a state_cache
    (kda_state_store; S may be prefill_snap's S_snap with slots.numel() states).  Slots outside the
    cache are skipped; of entries that name the same slot the last one is stored."""
    nslots, H, dk, dv, dev = _cache_args(cache, scales, slots)
    n = slots.numel()
    if S.dim() < 3 or tuple(S.shape[-3:]) != (H, dk, dv) or S.numel() != n * H * dk * dv:
        raise KdaError(f"S has shape {tuple(S.shape)}, expected {n} states of {(H, dk, dv)}")
    _dense(S, "S", torch.float32, S.shape, dev)
    rc = load().kda_state_store(_ptr(S), _ptr(slots), _ptr(cache), _ptr(scales), n, nslots, H, dk, dv,
                                _CACHE[cache.dtype], _stream())
    _check(rc, "kda_state_store")


def state_load(cache, scales, slots, S=None) -> torch.Tensor:
    """States [n,H,dk,dv] fp32 of the entries slots [n] int32 of a state_cache (zeros for slots
    outside it)."""
    nslots, H, dk, dv, dev = _cache_args(cache, scales, slots)
    n = slots.numel()
    if S is None:
        S = torch.empty(n, H, dk, dv, dtype=torch.float32, device=cache.device)
    _dense(S, "S", torch.float32, (n, H, dk, dv), dev)
    rc = load().kda_state_load(_ptr(cache), _ptr(scales), _ptr(slots), _ptr(S), n, nslots, H, dk, dv,
                               _CACHE[cache.dtype], _stream())
    _check(rc, "kda_state_load")
    return S
