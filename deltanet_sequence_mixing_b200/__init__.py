"""B200 (sm_100a) delta-rule sequence mixing: Python binding of the C ABI.

The functions below carry the names of the C entry points in
``include/deltanet.h`` and only marshal arguments: torch supplies device
memory and the current stream, and every step of the computation runs in the
library's CUDA kernels.  There is no CPU fallback.

    o, S = deltanet_chunk_fwd(q, k, v, beta, alpha=None, S0=None, C=64, prestep=False)
    o    = deltanet_decode_step(q, k, v, beta, S, alpha=None, prestep=False)  # S in place
    o, S, z = linear_attn_fwd(q, k, v, S0=None, z0=None, C=64)
    o, S = gated_linear_attn_fwd(q, k, v, alpha=None, S0=None)
    g    = gated_linear_attn_bwd(q, k, v, dO, alpha=None, S0=None, dS_T=None)
    o    = gated_linear_attn_decode_step(q, k, v, S, alpha=None)  # S in place
    q, k = qk_norm_rope_fwd(q, k, q_weight, k_weight, positions, inv_freq)
    g    = qk_norm_rope_bwd(q, k, dq, dk, q_weight, k_weight, positions, inv_freq)
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import _lib
from ._lib import DeltaNetError, check, lib, status_string  # noqa: F401

__all__ = [
    "deltanet_chunk_fwd", "deltanet_chunk_fwd_host", "deltanet_decode_step", "linear_attn_fwd",
    "deltanet_chunk_bwd", "seq_segments",
    "gated_linear_attn_fwd", "gated_linear_attn_bwd", "gated_linear_attn_decode_step",
    "qk_norm_rope_fwd", "qk_norm_rope_bwd",
    "workspace_for", "host_workspace_for",
    "deltanet_get_device_status", "deltanet_selftest_wait_timeout", "deltanet_selftest_wait_polls",
    "DeltaNetError",
]

_DT = {torch.float32: _lib.DN_F32, torch.bfloat16: _lib.DN_BF16}
_workspaces: dict = {}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _indexed(device) -> torch.device:
    """The device with its index: "cuda" is the current one, not one of its own."""
    device = torch.device("cuda" if device is None else device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


def workspace_for(device, nbytes: int = 256) -> torch.Tensor:
    """A cleared device workspace of at least ``nbytes``, cached per device; a
    larger one in its place takes over the status."""
    device = _indexed(device)
    ws = _workspaces.get(device)
    if ws is None or ws.numel() < nbytes:
        before, ws = ws, torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        check("deltanet_workspace_init",
              lib().deltanet_workspace_init(_ptr(ws), ws.numel(), _stream(device)))
        if before is not None:
            ws[:256].copy_(before[:256])
        _workspaces[device] = ws
    return ws


def _ws_bytes(B, H, T, Dk, Dv, C, dt):
    n = lib().deltanet_workspace_bytes(B, H, T, Dk, Dv, C, dt)
    if n == 0:
        raise DeltaNetError("deltanet_workspace_bytes", _lib.DN_ERR_UNSUPPORTED)
    return n


def _options(prestep, alpha, per_dim_rank):
    opts = _lib.DN_OPT_PRESTEP if prestep else 0
    if alpha is not None and alpha.dim() == per_dim_rank:
        opts |= _lib.DN_OPT_GATE_PER_DIM
    return opts


def deltanet_chunk_fwd(q, k, v, beta, alpha=None, S0=None, C: int = 64, o=None, S_out=None,
                       workspace=None, prestep: bool = False, seq_split: bool = False):
    """Chunkwise DeltaNet forward.  q, k: (B,H,T,Dk); v: (B,H,T,Dv) (bf16 or f32);
    beta: (B,H,T) f32; alpha: (B,H,T) f32 (one decay per token) or (B,H,T,Dk)
    (one per key dimension); S0: (B,H,Dk,Dv) f32.  ``prestep``: q, k are raw
    projections and beta logits (silu + L2 normalise and sigmoid run inside).
    ``seq_split``: permission to run each sequence as segments side by side
    (DN_OPT_SEQ_SPLIT; see seq_segments).  Returns (o, S_out)."""
    _need(q, "q")
    dev, dtype = q.device, q.dtype
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    for t, n in ((k, "k"), (v, "v")):
        _need(t, n, dtype, dev)
    _need(beta, "beta", torch.float32, dev)
    if alpha is not None:
        _need(alpha, "alpha", torch.float32, dev)
    if S0 is not None:
        _need(S0, "S0", torch.float32, dev)
    B, H, T, Dk = q.shape
    Dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, H, T, Dv, dtype=dtype, device=dev)
    if S_out is None:
        S_out = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev)
    _need(o, "o", dtype, dev)
    _need(S_out, "S_out", torch.float32, dev)
    dt = _DT[dtype]
    opts = _options(prestep, alpha, 4) | (_lib.DN_OPT_SEQ_SPLIT if seq_split else 0)
    nb = lib().deltanet_workspace_bytes_ex(B, H, T, Dk, Dv, C, dt, opts)
    if nb == 0:
        raise DeltaNetError("deltanet_workspace_bytes_ex", _lib.DN_ERR_UNSUPPORTED)
    ws = workspace if workspace is not None else workspace_for(dev, nb)
    if opts == 0:
        check("deltanet_chunk_fwd", lib().deltanet_chunk_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(S0), _ptr(o), _ptr(S_out),
            B, H, T, Dk, Dv, C, dt, _ptr(ws), ws.numel(), _stream(dev)))
    else:
        check("deltanet_chunk_fwd_ex", lib().deltanet_chunk_fwd_ex(
            _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(S0), _ptr(o), _ptr(S_out),
            B, H, T, Dk, Dv, C, dt, opts, _ptr(ws), ws.numel(), _stream(dev)))
    return o, S_out


def seq_segments(B, H, T, Dk, Dv, C=64, dtype=torch.bfloat16, prestep=False, per_dim=False,
                 seq_split=True) -> int:
    """Segments a deltanet_chunk_fwd call with these arguments runs on the
    current device (1: the sequence is not split)."""
    opts = (_lib.DN_OPT_PRESTEP if prestep else 0) | (_lib.DN_OPT_GATE_PER_DIM if per_dim else 0) | (
        _lib.DN_OPT_SEQ_SPLIT if seq_split else 0)
    return int(lib().deltanet_seq_segments(B, H, T, Dk, Dv, C, _DT[dtype], opts))


def deltanet_chunk_bwd(q, k, v, beta, dO, alpha=None, S0=None, dS_T=None, workspace=None):
    """Gradient of deltanet_chunk_fwd for the loss sum(dO * o) + sum(dS_T * S_T).
    Returns dict(dq, dk, dv, dbeta, dlog_alpha, dS0), float32 tensors
    (dlog_alpha is None when ungated)."""
    _need(q, "q")
    dev, dtype = q.device, q.dtype
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    for t, n in ((k, "k"), (v, "v"), (dO, "dO")):
        _need(t, n, dtype, dev)
    _need(beta, "beta", torch.float32, dev)
    for t, n in ((alpha, "alpha"), (S0, "S0"), (dS_T, "dS_T")):
        if t is not None:
            _need(t, n, torch.float32, dev)
    B, H, T, Dk = q.shape
    Dv = v.shape[-1]
    f = dict(dtype=torch.float32, device=dev)
    out = dict(dq=torch.empty(B, H, T, Dk, **f), dk=torch.empty(B, H, T, Dk, **f),
               dv=torch.empty(B, H, T, Dv, **f), dbeta=torch.empty(B, H, T, **f),
               dlog_alpha=None if alpha is None else torch.empty(B, H, T, **f),
               dS0=torch.empty(B, H, Dk, Dv, **f))
    nb = lib().deltanet_chunk_bwd_workspace_bytes(B, H, T, Dk, Dv, _DT[dtype])
    if nb == 0:
        raise DeltaNetError("deltanet_chunk_bwd_workspace_bytes", _lib.DN_ERR_UNSUPPORTED)
    ws = workspace if workspace is not None else torch.empty(nb, dtype=torch.uint8, device=dev)
    check("deltanet_chunk_bwd", lib().deltanet_chunk_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(S0), _ptr(dO), _ptr(dS_T),
        _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dbeta"]),
        _ptr(out["dlog_alpha"]), _ptr(out["dS0"]), B, H, T, Dk, Dv, _DT[dtype], _ptr(ws), ws.numel(),
        _stream(dev)))
    return out


def _need_host(t, name, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.is_cuda:
        raise ValueError(f"{name} must be a host tensor for the host-buffer call")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def host_workspace_for(device, B, H, T, Dk, Dv, C, dtype) -> torch.Tensor:
    """A device workspace for deltanet_chunk_fwd_host (cleared, not cached)."""
    device = torch.device(device)
    nb = lib().deltanet_host_workspace_bytes(B, H, T, Dk, Dv, C, _DT[dtype])
    if nb == 0:
        raise DeltaNetError("deltanet_host_workspace_bytes", _lib.DN_ERR_UNSUPPORTED)
    ws = torch.empty(nb, dtype=torch.uint8, device=device)
    check("deltanet_workspace_init", lib().deltanet_workspace_init(_ptr(ws), ws.numel(), _stream(device)))
    return ws


def deltanet_chunk_fwd_host(q, k, v, beta, alpha=None, S0=None, C: int = 64, o=None, S_out=None,
                            workspace=None, device=None):
    """deltanet_chunk_fwd on host tensors (page-locked for overlapped copies):
    the heads stream through the device in groups, copies overlapping the
    compute.  Asynchronous on the device's current stream: synchronize it
    before reading (o, S_out)."""
    _need_host(q, "q")
    dtype = q.dtype
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    for t, n in ((k, "k"), (v, "v")):
        _need_host(t, n, dtype)
    _need_host(beta, "beta", torch.float32)
    for t, n in ((alpha, "alpha"), (S0, "S0")):
        if t is not None:
            _need_host(t, n, torch.float32)
    B, H, T, Dk = q.shape
    Dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, H, T, Dv, dtype=dtype).pin_memory()
    if S_out is None:
        S_out = torch.empty(B, H, Dk, Dv, dtype=torch.float32).pin_memory()
    _need_host(o, "o", dtype)
    _need_host(S_out, "S_out", torch.float32)
    device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    if workspace is None:
        workspace = host_workspace_for(device, B, H, T, Dk, Dv, C, dtype)
    _need(workspace, "workspace", torch.uint8, device)
    with torch.cuda.device(device):
        check("deltanet_chunk_fwd_host", lib().deltanet_chunk_fwd_host(
            _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(S0), _ptr(o), _ptr(S_out),
            B, H, T, Dk, Dv, C, _DT[dtype], _ptr(workspace), workspace.numel(), _stream(device)))
    return o, S_out


def linear_attn_fwd(q, k, v, S0=None, z0=None, C: int = 64, o=None, S_out=None, z_out=None,
                    workspace=None):
    """Chunkwise ELU+1 causal linear attention.  Returns (o, S_out, z_out)."""
    _need(q, "q")
    dev, dtype = q.device, q.dtype
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    for t, n in ((k, "k"), (v, "v")):
        _need(t, n, dtype, dev)
    for t, n in ((S0, "S0"), (z0, "z0")):
        if t is not None:
            _need(t, n, torch.float32, dev)
    B, H, T, Dk = q.shape
    Dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, H, T, Dv, dtype=dtype, device=dev)
    if S_out is None:
        S_out = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev)
    if z_out is None:
        z_out = torch.empty(B, H, Dk, dtype=torch.float32, device=dev)
    dt = _DT[dtype]
    nb = _ws_bytes(B, H, T, Dk, Dv, C, dt)
    ws = workspace if workspace is not None else workspace_for(dev, nb)
    check("linear_attn_fwd", lib().linear_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(S0), _ptr(z0), _ptr(o), _ptr(S_out), _ptr(z_out),
        B, H, T, Dk, Dv, C, dt, _ptr(ws), ws.numel(), _stream(dev)))
    return o, S_out, z_out


def deltanet_decode_step(q, k, v, beta, S, alpha=None, o=None, prestep: bool = False):
    """One decode step.  q, k: (B,H,Dk); v: (B,H,Dv); beta: (B,H) f32; alpha:
    (B,H) f32 or (B,H,Dk) (one decay per key dimension); S: (B,H,Dk,Dv) f32,
    updated in place.  ``prestep``: q, k raw and beta logits.  Returns o (B,H,Dv)."""
    _need(q, "q")
    dev, dtype = q.device, q.dtype
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    for t, n in ((k, "k"), (v, "v")):
        _need(t, n, dtype, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(S, "S", torch.float32, dev)
    if alpha is not None:
        _need(alpha, "alpha", torch.float32, dev)
    B, H, Dk = q.shape
    Dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, H, Dv, dtype=dtype, device=dev)
    opts = _options(prestep, alpha, 3)
    if opts == 0:
        check("deltanet_decode_step", lib().deltanet_decode_step(
            _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(S), _ptr(o),
            B, H, Dk, Dv, _DT[dtype], _stream(dev)))
    else:
        check("deltanet_decode_step_ex", lib().deltanet_decode_step_ex(
            _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(S), _ptr(o),
            B, H, Dk, Dv, _DT[dtype], opts, _stream(dev)))
    return o


# The calls below serve single tokens too, where the host's time is the call's:
# checks take one short path when nothing is wrong, addresses go to ctypes as
# integers, and a call for another device than the current one starts over there.
_current_device = torch._C._cuda_getDevice
_current_raw_stream = torch._C._cuda_getCurrentRawStream


def _at(t):
    return None if t is None else t.data_ptr()


def _need_shape(t, name, shape, dtype, device, optional=False):
    """A contiguous tensor of this shape, type and device (or None)."""
    if t is None and optional:
        return None
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.shape == shape
            and t.is_contiguous()):
        return t
    _need(t, name, dtype, device)
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


_stream_workspaces: dict = {}
_scratch_devices: set = set()  # devices with calls that had scratch, on whatever stream
_scratch_call = threading.Lock()  # a call's launches go together: threads may share a stream, and so its scratch
_KEEP_BYTES = 32 << 20  # larger scratch is allocated for each call


def _own_workspace(device, nbytes: int) -> torch.Tensor:
    """The workspace of a call that brings none.  Without scratch it is the
    device's cached status word (kernels only ever set bits in it).  Scratch is
    kept for each stream, whose calls follow one another; under graph capture,
    or where it is large, it comes from the caching allocator for this call
    alone, so two graphs or two streams never share it.  Nobody reads the status
    word in scratch: a timeout is in the device's own word, too."""
    capturing = torch.cuda.is_current_stream_capturing()
    if nbytes <= 256 and not capturing:
        return workspace_for(device)
    stream = _current_raw_stream(device.index)
    keep = nbytes <= _KEEP_BYTES and not capturing
    ws = _stream_workspaces.get((device.index, stream)) if keep else None
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _scratch_devices.add(device.index)
        if keep:
            _stream_workspaces[(device.index, stream)] = ws
    return ws


def _recurrence_inputs(q, k, v, alpha, rank):
    """Device, type and sizes of a gated recurrence call, its inputs checked."""
    _need(q, "q")
    dev, dtype = q.device, q.dtype
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    shape = q.shape
    if len(shape) != rank:
        raise ValueError(f"q must have {rank} dimensions, got {len(shape)}")
    _need_shape(k, "k", shape, dtype, dev)
    if not isinstance(v, torch.Tensor):
        raise TypeError("v must be a torch.Tensor")
    if v.dim() != rank:
        raise ValueError(f"v must have {rank} dimensions, got {v.dim()}")
    lead, Dv = shape[:-1], v.shape[-1]
    _need_shape(v, "v", (*lead, Dv), dtype, dev)
    _need_shape(alpha, "alpha", lead, torch.float32, dev, True)
    return dev, dtype, lead, shape[-1], Dv


def _gated_bytes(fn, B, H, T, Dk, Dv, dtype):
    n = getattr(lib(), fn)(B, H, T, Dk, Dv, _DT[dtype])
    if n == 0:
        raise DeltaNetError(fn, _lib.DN_ERR_UNSUPPORTED)
    return n


def gated_linear_attn_fwd(q, k, v, alpha=None, S0=None, o=None, S_out=None, workspace=None):
    """Gated linear recurrence S_t = alpha_t S_{t-1} + k_t^T v_t, o_t = q_t S_t.
    q, k: (B,H,T,Dk); v: (B,H,T,Dv) (bf16 or f32); alpha: (B,H,T) f32 in [0,1]
    or None (1); S0: (B,H,Dk,Dv) f32 or None (0).  S_out may be S0.  Returns
    (o, S_out): (B,H,T,Dv) of q's type and (B,H,Dk,Dv) f32."""
    dev, dtype, (B, H, T), Dk, Dv = _recurrence_inputs(q, k, v, alpha, 4)
    _need_shape(S0, "S0", (B, H, Dk, Dv), torch.float32, dev, True)
    _need_shape(o, "o", (B, H, T, Dv), dtype, dev, True)
    _need_shape(S_out, "S_out", (B, H, Dk, Dv), torch.float32, dev, True)
    if _current_device() != dev.index:
        with torch.cuda.device(dev):
            return gated_linear_attn_fwd(q, k, v, alpha, S0, o, S_out, workspace)
    if o is None:
        o = torch.empty_like(v)
    if S_out is None:
        S_out = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev)
    with _scratch_call:
        if workspace is None:
            ws = _own_workspace(dev, _gated_bytes("gated_linear_attn_workspace_bytes", B, H, T, Dk, Dv, dtype))
        else:
            ws = _need(workspace, "workspace", torch.uint8, dev)
        check("gated_linear_attn_fwd", lib().gated_linear_attn_fwd(
            _at(q), _at(k), _at(v), _at(alpha), _at(S0), _at(o), _at(S_out),
            B, H, T, Dk, Dv, _DT[dtype], _at(ws), ws.numel(), _current_raw_stream(dev.index)))
    return o, S_out


def gated_linear_attn_bwd(q, k, v, dO, alpha=None, S0=None, dS_T=None, workspace=None):
    """Gradient of gated_linear_attn_fwd for the loss sum(dO * o) + sum(dS_T * S_T).
    Returns dict(dq, dk, dv, dlog_alpha, dS0): dq, dk, dv of q's type (summed in
    float32, rounded once), dlog_alpha (None when ungated) and dS0 float32."""
    dev, dtype, (B, H, T), Dk, Dv = _recurrence_inputs(q, k, v, alpha, 4)
    _need_shape(dO, "dO", (B, H, T, Dv), dtype, dev)
    for t, n in ((S0, "S0"), (dS_T, "dS_T")):
        _need_shape(t, n, (B, H, Dk, Dv), torch.float32, dev, True)
    if _current_device() != dev.index:
        with torch.cuda.device(dev):
            return gated_linear_attn_bwd(q, k, v, dO, alpha, S0, dS_T, workspace)
    f = dict(dtype=torch.float32, device=dev)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dlog_alpha=None if alpha is None else torch.empty(B, H, T, **f),
               dS0=torch.empty(B, H, Dk, Dv, **f))
    with _scratch_call:
        if workspace is None:
            ws = _own_workspace(dev, _gated_bytes("gated_linear_attn_bwd_workspace_bytes", B, H, T, Dk, Dv, dtype))
        else:
            ws = _need(workspace, "workspace", torch.uint8, dev)
        check("gated_linear_attn_bwd", lib().gated_linear_attn_bwd(
            _at(q), _at(k), _at(v), _at(alpha), _at(S0), _at(dO), _at(dS_T), _at(out["dq"]),
            _at(out["dk"]), _at(out["dv"]), _at(out["dlog_alpha"]), _at(out["dS0"]),
            B, H, T, Dk, Dv, _DT[dtype], _at(ws), ws.numel(), _current_raw_stream(dev.index)))
    return out


def gated_linear_attn_decode_step(q, k, v, S, alpha=None, o=None):
    """One token of the gated linear recurrence for every cached state.  q, k:
    (B,H,Dk); v: (B,H,Dv); alpha: (B,H) f32 or None; S: (B,H,Dk,Dv) f32, updated
    in place.  Returns o (B,H,Dv) of q's type."""
    dev, dtype, (B, H), Dk, Dv = _recurrence_inputs(q, k, v, alpha, 3)
    _need_shape(S, "S", (B, H, Dk, Dv), torch.float32, dev)
    _need_shape(o, "o", (B, H, Dv), dtype, dev, True)
    if _current_device() != dev.index:
        with torch.cuda.device(dev):
            return gated_linear_attn_decode_step(q, k, v, S, alpha, o)
    if o is None:
        o = torch.empty_like(v)
    check("gated_linear_attn_decode_step", lib().gated_linear_attn_decode_step(
        _at(q), _at(k), _at(v), _at(alpha), _at(S), _at(o), B, H, Dk, Dv, _DT[dtype], _current_raw_stream(dev.index)))
    return o


def _need_rows(t, name, dtype=None, device=None):
    """A (B,T,H,D) tensor, strided, with contiguous rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dim() != 4:
        raise ValueError(f"{name} must have 4 dimensions (B,T,H,D), got {t.dim()}")
    if t.stride(3) != 1 and t.numel() > 0:
        raise ValueError(f"{name} must have contiguous rows")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _row_strides(t):
    """Strides over b, t and h; an axis of one element or none has stride 0."""
    sb, st, sh, _ = t.stride()
    B, T, H, _ = t.shape
    return sb if B > 1 else 0, st if T > 1 else 0, sh if H > 1 else 0


def _qk_args(q, k, q_weight, k_weight, positions, inv_freq, norm, eps, silu, interleaved):
    _need_rows(q, "q")
    dev, dtype = q.device, q.dtype
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    _need_rows(k, "k", dtype, dev)
    B, T, Hq, D = q.shape
    Hk = k.shape[2]
    if k.shape != (B, T, Hk, D):
        raise ValueError(f"k must have shape {(B, T, 'Hk', D)}, got {tuple(k.shape)}")
    for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        _need_shape(t, n, (D,), torch.float32, dev, True)
    pos_stride = 0
    if positions is not None:
        _need(positions, "positions", torch.int64, dev)
        if positions.shape == (B, T):
            pos_stride = T
        elif positions.shape != (T,):
            raise ValueError(f"positions must have shape {(B, T)} or {(T,)}, got {tuple(positions.shape)}")
    rot = 0
    if inv_freq is not None:
        _need(inv_freq, "inv_freq", torch.float32, dev)
        if inv_freq.dim() != 1:
            raise ValueError(f"inv_freq must have one dimension, got {inv_freq.dim()}")
        rot = 2 * inv_freq.shape[0]
    if norm not in ("rms", "l2"):
        raise ValueError(f'norm must be "rms" or "l2", got {norm!r}')
    if eps is None:
        eps = 1e-6 if norm == "rms" else 1e-12
    opts = ((_lib.DN_QK_L2 if norm == "l2" else 0) | (_lib.DN_QK_SILU if silu else 0)
            | (_lib.DN_QK_INTERLEAVED if interleaved else 0))
    return dev, dtype, B, T, Hq, Hk, D, rot, pos_stride, float(eps), opts


def qk_norm_rope_fwd(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, norm: str = "rms",
                     eps=None, silu: bool = False, interleaved: bool = False, q_out=None, k_out=None):
    """Per-head norm of queries and keys and their rotation by position.
    q: (B,T,Hq,D), k: (B,T,Hk,D), strided views with contiguous rows (bf16 or
    f32, bases and strides multiples of 16 bytes); weights: (D,) f32 or None;
    positions: (B,T) or (T,) int64, None for 0..T-1; inv_freq: (rot/2,) f32,
    None for no rotation; norm: "rms" (eps 1e-6 inside the root) or "l2" (the
    norm at least eps, 1e-12); ``silu``: the feature map in front of the norm;
    ``interleaved``: pairs (2i, 2i+1) instead of (i, i + rot/2).  Returns
    (B,Hq,T,D) and (B,Hk,T,D), contiguous: what the mixing calls take."""
    dev, dtype, B, T, Hq, Hk, D, rot, ps, eps, opts = _qk_args(
        q, k, q_weight, k_weight, positions, inv_freq, norm, eps, silu, interleaved)
    _need_shape(q_out, "q_out", (B, Hq, T, D), dtype, dev, True)
    _need_shape(k_out, "k_out", (B, Hk, T, D), dtype, dev, True)
    if _current_device() != dev.index:
        with torch.cuda.device(dev):
            return qk_norm_rope_fwd(q, k, q_weight, k_weight, positions, inv_freq, norm, eps, silu, interleaved,
                                    q_out, k_out)
    if q_out is None:
        q_out = torch.empty(B, Hq, T, D, dtype=dtype, device=dev)
    if k_out is None:
        k_out = torch.empty(B, Hk, T, D, dtype=dtype, device=dev)
    check("qk_norm_rope_fwd", lib().qk_norm_rope_fwd(
        _at(q), _at(k), _at(q_weight), _at(k_weight), _at(positions), _at(inv_freq), _at(q_out),
        _at(k_out), B, T, Hq, Hk, D, rot, *_row_strides(q), *_row_strides(k), ps, eps, opts, _DT[dtype],
        _current_raw_stream(dev.index)))
    return q_out, k_out


def qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, positions=None, inv_freq=None,
                     norm: str = "rms", eps=None, silu: bool = False, interleaved: bool = False, dq=None, dk=None,
                     workspace=None):
    """Gradient of qk_norm_rope_fwd.  dq_out: (B,Hq,T,D) and dk_out: (B,Hk,T,D),
    both of q's type or both float32; dq, dk: where to write the derivatives by q and k
    ((B,T,H,D) views like q and k, slices of one fused gradient, say; new
    tensors if None).  Returns dict(dq, dk, dq_weight, dk_weight), the weights'
    derivatives (D,) float32, None for a weight that is None."""
    dev, dtype, B, T, Hq, Hk, D, rot, ps, eps, opts = _qk_args(
        q, k, q_weight, k_weight, positions, inv_freq, norm, eps, silu, interleaved)
    if not isinstance(dq_out, torch.Tensor) or not isinstance(dk_out, torch.Tensor):
        raise TypeError("dq_out and dk_out must be torch.Tensors")
    gdt = dq_out.dtype
    if gdt not in (dtype, torch.float32):
        raise TypeError(f"dq_out must be {dtype} or torch.float32, got {gdt}")
    _need_shape(dq_out, "dq_out", (B, Hq, T, D), gdt, dev)
    _need_shape(dk_out, "dk_out", (B, Hk, T, D), gdt, dev)
    if _current_device() != dev.index:
        with torch.cuda.device(dev):
            return qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight, k_weight, positions, inv_freq, norm, eps, silu,
                                    interleaved, dq, dk, workspace)
    if dq is None:
        dq = torch.empty(B, T, Hq, D, dtype=dtype, device=dev)
    if dk is None:
        dk = torch.empty(B, T, Hk, D, dtype=dtype, device=dev)
    for t, n, like in ((dq, "dq", q), (dk, "dk", k)):
        _need_rows(t, n, dtype, dev)
        if t.shape != like.shape:
            raise ValueError(f"{n} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
    dw = [None if w is None else torch.empty(D, dtype=torch.float32, device=dev) for w in (q_weight, k_weight)]
    ws = workspace
    if ws is None and (q_weight is not None or k_weight is not None):
        nb = lib().qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hk, D)
        if nb == 0:
            raise DeltaNetError("qk_norm_rope_bwd_workspace_bytes", _lib.DN_ERR_UNSUPPORTED)
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    if ws is not None:
        _need(ws, "workspace", torch.uint8, dev)
    check("qk_norm_rope_bwd", lib().qk_norm_rope_bwd(
        _at(q), _at(k), _at(dq_out), _at(dk_out), _at(q_weight), _at(k_weight), _at(positions),
        _at(inv_freq), _at(dq), _at(dk), _at(dw[0]), _at(dw[1]), B, T, Hq, Hk, D, rot,
        *_row_strides(q), *_row_strides(k), *_row_strides(dq), *_row_strides(dk), ps, eps, opts, _DT[dtype],
        _DT[gdt], _at(ws), 0 if ws is None else ws.numel(), _current_raw_stream(dev.index)))
    return dict(dq=dq, dk=dk, dq_weight=dw[0], dk_weight=dw[1])


def deltanet_get_device_status(device=None, workspace=None) -> int:
    """Synchronise and return the sticky device status of ``workspace``, or of
    ``device``: of its cached workspace and, whatever workspace they had, of the
    gated recurrence's calls on all of its streams."""
    device = _indexed(device)
    if workspace is not None:
        return lib().deltanet_get_device_status(_ptr(workspace), _stream(device))
    status = lib().deltanet_get_device_status(_ptr(workspace_for(device)), _stream(device))
    if status == 0:
        if device.index in _scratch_devices:
            torch.cuda.synchronize(device)  # their streams may be gone by now
        with torch.cuda.device(device):
            status = lib().deltanet_get_recurrence_status(_stream(device))
    return status


def deltanet_selftest_wait_timeout(wait_ns: int, workspace, device=None) -> int:
    """Launch the bounded-wait self test on ``workspace``; returns the launch status."""
    device = torch.device(device if device is not None else workspace.device)
    return lib().deltanet_selftest_wait_timeout(_ptr(workspace), workspace.numel(), int(wait_ns),
                                                _stream(device))


def deltanet_selftest_wait_polls(polls: int, workspace, device=None) -> int:
    """The bounded-wait self test of the gated recurrence's kernels, whose waits
    count polls; returns the launch status."""
    device = torch.device(device if device is not None else workspace.device)
    return lib().deltanet_selftest_wait_polls(_ptr(workspace), workspace.numel(), int(polls), _stream(device))


def reset_device_status(device=None, workspace=None) -> None:
    """Clear the status of ``workspace`` (or all that the query of ``device`` reads)."""
    device = _indexed(device)
    ws = workspace if workspace is not None else workspace_for(device)
    check("deltanet_workspace_init", lib().deltanet_workspace_init(_ptr(ws), ws.numel(), _stream(device)))
    if workspace is None:
        if device.index in _scratch_devices:
            torch.cuda.synchronize(device)  # a call in flight on another stream comes before the reset
        with torch.cuda.device(device):
            check("deltanet_clear_recurrence_status", lib().deltanet_clear_recurrence_status(_stream(device)))
