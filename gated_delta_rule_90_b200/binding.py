"""ctypes binding of libgdr (include/gdr.h) for torch tensors.

Argument marshalling only: shapes are read off the tensors, outputs and the
workspace are allocated with torch, and every step of the computation runs
in libgdr's CUDA kernels.  There is no fallback: if the library is missing
the call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdr.so")
# The checked build (kernels guard their accesses; see gdr.h, gdr_checked_build).
CHECKED_LIB_PATH = os.path.join(_HERE, "libgdr_check.so")
# GDR_LIBRARY=<path> loads another build of the same library instead, e.g.
# CHECKED_LIB_PATH.
LIB_ENV = "GDR_LIBRARY"

GDR_OK, GDR_ERR_INVALID, GDR_ERR_UNSUPPORTED, GDR_ERR_CUDA, GDR_ERR_TIMEOUT, GDR_ERR_BOUNDS = \
    range(6)
GDR_F32, GDR_BF16 = 0, 1
GDR_GATE_SCALAR, GDR_GATE_PER_KEY_CHANNEL, GDR_GATE_HEAD = 0, 1, 2
PATHS = {"auto": 0, "simt": 1, "tc": 2}
KERNELS = {"decode": 0, "fwd_simt": 1, "tc_plan": 2, "tc_wy": 3, "tc_state": 4, "gdp_remap": 5,
           "gdn2_simt": 6, "gdn2_decode": 7, "frame_gram": 8, "frame_solve": 9, "frame_chain": 10,
           "frame_out": 11, "lin_decode": 12, "lin_plan": 13, "lin_state": 14, "lin_scan": 15,
           "lin_out": 16, "lin_grad": 17, "lin_sum": 18}

_lib = None


class GdrError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def library_path() -> str:
    """The library lib() loads: $GDR_LIBRARY if set, else libgdr.so."""
    return os.environ.get(LIB_ENV) or LIB_PATH


def lib() -> ctypes.CDLL:
    """Load libgdr.so (built in-tree by __graft_entry__.build())."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{os.path.basename(path)} is not built ({path}); "
                               "run __graft_entry__.build()")
        L = ctypes.CDLL(path)
        vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.gdr_status_string.restype = ctypes.c_char_p
        L.gdr_status_string.argtypes = [i]
        L.gdr_fwd_workspace_size.restype = sz
        L.gdr_fwd_workspace_size.argtypes = [i, i, i, i, i, i, i, i, i, i, i]
        L.gdr_fwd.restype = i
        L.gdr_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, i, i, i, i,
                              vp, sz, vp]
        L.gdr_decode_step.restype = i
        L.gdr_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
        L.gdr_device_status.restype = i
        L.gdr_device_status.argtypes = [vp]
        L.gdr_selftest_wait_timeout.restype = i
        L.gdr_selftest_wait_timeout.argtypes = [ctypes.c_uint, vp]
        L.gdr_checked_build.restype = i
        L.gdr_checked_build.argtypes = []
        L.gdr_selftest_bounds.restype = i
        L.gdr_selftest_bounds.argtypes = [vp]
        L.gdr_fwd_product_workspace_size.restype = sz
        L.gdr_fwd_product_workspace_size.argtypes = [i] * 12
        L.gdr_fwd_product.restype = i
        L.gdr_fwd_product.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, i,
                                      i, i, i, vp, sz, vp]
        L.gdr_fwd_gdn2.restype = i
        L.gdr_fwd_gdn2.argtypes = [vp] * 9 + [i] * 6 + [vp, i, i, i, i, vp, sz, vp]
        L.gdr_fwd_gdn2_workspace_size.restype = sz
        L.gdr_fwd_gdn2_workspace_size.argtypes = [i] * 11
        L.gdr_decode_step_gdn2.restype = i
        L.gdr_decode_step_gdn2.argtypes = [vp] * 8 + [i] * 6 + [vp]
        L.gdr_fwd_frame_workspace_size.restype = sz
        L.gdr_fwd_frame_workspace_size.argtypes = [i] * 6
        L.gdr_fwd_frame.restype = i
        L.gdr_fwd_frame.argtypes = [vp] * 8 + [i] * 8 + [vp, sz, vp]
        L.gdr_fwd_linear_workspace_size.restype = sz
        L.gdr_fwd_linear_workspace_size.argtypes = [i] * 11
        L.gdr_fwd_linear.restype = i
        L.gdr_fwd_linear.argtypes = [vp] * 7 + [i] * 6 + [vp, i, i, i, i, vp, sz, vp]
        L.gdr_decode_step_linear.restype = i
        L.gdr_decode_step_linear.argtypes = [vp] * 6 + [i] * 7 + [vp]
        L.gdr_bwd_linear_workspace_size.restype = sz
        L.gdr_bwd_linear_workspace_size.argtypes = [i] * 11
        L.gdr_bwd_linear.restype = i
        L.gdr_bwd_linear.argtypes = [vp] * 12 + [i] * 6 + [vp, i, i, i, i, vp, sz, vp]
        L.gdr_profile_enable.restype = None
        L.gdr_profile_enable.argtypes = [i]
        L.gdr_profile_read.restype = i
        L.gdr_profile_read.argtypes = [i, ctypes.POINTER(ctypes.c_longlong),
                                       ctypes.POINTER(ctypes.c_double)]
        L.gdr_set_gram_spread_limit.restype = ctypes.c_float
        L.gdr_set_gram_spread_limit.argtypes = [ctypes.c_float]
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().gdr_status_string(int(status)).decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device=None) -> ctypes.c_void_p:
    """The cudaStream_t handle of ``stream`` (None: the current stream of
    ``device``).  A torch stream must belong to ``device``: the library
    launches on the current device, which the calls below set to it."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    sdev = getattr(stream, "device", None)
    if device is not None and sdev is not None and torch.device(sdev) != torch.device(device):
        raise ValueError(f"stream belongs to {sdev}; the tensors are on {device}")
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _call_on(device, fn):
    """Run ``fn`` with ``device`` as the current CUDA device.  libgdr launches
    on the current device (its tensor maps, error word and scratch lookup are
    per device), so every call is made with the tensors' device current."""
    with torch.cuda.device(device):
        return fn()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDR_BF16
    if t.dtype == torch.float32:
        return GDR_F32
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _need_contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _check(device, *specs):
    """The memory the kernels will read or write, checked before the call:
    each ``(name, tensor, dtype, numel)`` (tensor None = absent) must live on
    ``device``, have ``dtype`` (None: not checked) and hold at least ``numel``
    elements.  A tensor on another device, of a narrower type or too small
    would otherwise be addressed out of bounds by the kernels."""
    for name, t, dtype, numel in specs:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}; expected {device}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.numel() < numel:
            raise ValueError(f"{name} holds {t.numel()} elements; needs {numel}")


def _on_cuda(q):
    if not isinstance(q, torch.Tensor) or q.device.type != "cuda":
        raise ValueError("tensors must be CUDA tensors")
    return q.device


def fwd_workspace_size(B, T, H, d_k, d_v, chunk, n_seq, varlen, dtype, gate, path="auto") -> int:
    return int(lib().gdr_fwd_workspace_size(B, T, H, d_k, d_v, chunk, n_seq, int(bool(varlen)),
                                            dtype, gate, PATHS[path]))


def fwd_product_workspace_size(B, T, H, n_h, d_k, d_v, chunk, n_seq, varlen, dtype, gate,
                               path="auto") -> int:
    return int(lib().gdr_fwd_product_workspace_size(B, T, H, n_h, d_k, d_v, chunk, n_seq,
                                                    int(bool(varlen)), dtype, gate, PATHS[path]))


def gdr_fwd(q, k, v, g, beta, S0=None, *, chunk: int = 64, cu_seqlens=None, out=None,
            S_final=None, want_final: bool = True, path: str = "auto", workspace=None,
            stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Prefill: returns ``(out [B,T,H,d_v], S_final [N,H,d_v,d_k] or None)``."""
    B, T, H, d_k = q.shape
    d_v = v.shape[-1]
    dtype = _dtype_code(q)
    gate = GDR_GATE_PER_KEY_CHANNEL if g.dim() == 4 else GDR_GATE_SCALAR
    n_seq = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    _need_contig(q, k, v, g, beta, S0, cu_seqlens)
    dev, th = _on_cuda(q), B * T * H
    _check(dev, ("k", k, q.dtype, th * d_k), ("v", v, q.dtype, th * d_v),
           ("g", g, torch.float32, th * (d_k if gate else 1)), ("beta", beta, torch.float32, th),
           ("S0", S0, torch.float32, n_seq * H * d_v * d_k), ("cu_seqlens", cu_seqlens, torch.int32, 1),
           ("out", out, q.dtype, th * d_v), ("S_final", S_final, torch.float32, n_seq * H * d_v * d_k))
    if out is None:
        out = torch.empty((B, T, H, d_v), dtype=q.dtype, device=q.device)
    if S_final is None and want_final:
        S_final = torch.empty((n_seq, H, d_v, d_k), dtype=torch.float32, device=q.device)
    ws_bytes = fwd_workspace_size(B, T, H, d_k, d_v, chunk, n_seq, cu_seqlens is not None, dtype,
                                  gate, path)
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    ws_avail = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(dev, ("workspace", workspace, None, 0))
    st = _call_on(dev, lambda: lib().gdr_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(out), _ptr(S_final), B, T,
        H, d_k, d_v, chunk, _ptr(cu_seqlens), n_seq, dtype, gate, PATHS[path], _ptr(workspace),
        ws_avail, _stream(stream, dev)))
    if st != GDR_OK:
        raise GdrError(st, "gdr_fwd")
    return out, S_final


def gdr_fwd_product(q, k, v, g, beta, S0=None, *, chunk: int = 64, cu_seqlens=None, out=None,
                    S_final=None, want_final: bool = True, path: str = "auto", workspace=None,
                    stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gated DeltaProduct prefill: k [B,T,n_h,H,d_k], v [B,T,n_h,H,d_v],
    beta [B,T,n_h,H]; returns (out [B,T,H,d_v], S_final)."""
    B, T, H, d_k = q.shape
    n_h = k.shape[2]
    d_v = v.shape[-1]
    dtype = _dtype_code(q)
    gate = GDR_GATE_PER_KEY_CHANNEL if g.dim() == 4 else GDR_GATE_SCALAR
    n_seq = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    _need_contig(q, k, v, g, beta, S0, cu_seqlens)
    dev, th = _on_cuda(q), B * T * H
    _check(dev, ("k", k, q.dtype, th * n_h * d_k), ("v", v, q.dtype, th * n_h * d_v),
           ("g", g, torch.float32, th * (d_k if gate else 1)),
           ("beta", beta, torch.float32, th * n_h),
           ("S0", S0, torch.float32, n_seq * H * d_v * d_k), ("cu_seqlens", cu_seqlens, torch.int32, 1),
           ("out", out, q.dtype, th * d_v), ("S_final", S_final, torch.float32, n_seq * H * d_v * d_k))
    if out is None:
        out = torch.empty((B, T, H, d_v), dtype=q.dtype, device=q.device)
    if S_final is None and want_final:
        S_final = torch.empty((n_seq, H, d_v, d_k), dtype=torch.float32, device=q.device)
    ws_bytes = int(lib().gdr_fwd_product_workspace_size(B, T, H, n_h, d_k, d_v, chunk, n_seq,
                                                       int(cu_seqlens is not None), dtype, gate,
                                                       PATHS[path]))
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    ws_avail = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(dev, ("workspace", workspace, None, 0))
    st = _call_on(dev, lambda: lib().gdr_fwd_product(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(out), _ptr(S_final), B, T,
        H, n_h, d_k, d_v, chunk, _ptr(cu_seqlens), n_seq, dtype, gate, PATHS[path],
        _ptr(workspace), ws_avail, _stream(stream, dev)))
    if st != GDR_OK:
        raise GdrError(st, "gdr_fwd_product")
    return out, S_final


def fwd_gdn2_workspace_size(B, T, H, d_k, d_v, chunk, n_seq, varlen, dtype, gate,
                            path="auto") -> int:
    return int(lib().gdr_fwd_gdn2_workspace_size(B, T, H, d_k, d_v, chunk, n_seq,
                                                 int(bool(varlen)), dtype, gate, PATHS[path]))


def gdr_fwd_gdn2(q, k, v, g, b, w, S0=None, *, chunk: int = 64, cu_seqlens=None, out=None,
                 S_final=None, want_final: bool = True, path: str = "auto", workspace=None,
                 stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gated DeltaNet-2 prefill: erase gate b [B,T,H,d_k], write gate w
    [B,T,H,d_v] (fp32); returns (out [B,T,H,d_v], S_final)."""
    B, T, H, d_k = q.shape
    d_v = v.shape[-1]
    dtype = _dtype_code(q)
    gate = GDR_GATE_PER_KEY_CHANNEL if g.dim() == 4 else GDR_GATE_SCALAR
    n_seq = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    _need_contig(q, k, v, g, b, w, S0, cu_seqlens)
    dev, th = _on_cuda(q), B * T * H
    _check(dev, ("k", k, q.dtype, th * d_k), ("v", v, q.dtype, th * d_v),
           ("g", g, torch.float32, th * (d_k if gate else 1)), ("b", b, torch.float32, th * d_k),
           ("w", w, torch.float32, th * d_v),
           ("S0", S0, torch.float32, n_seq * H * d_v * d_k), ("cu_seqlens", cu_seqlens, torch.int32, 1),
           ("out", out, q.dtype, th * d_v), ("S_final", S_final, torch.float32, n_seq * H * d_v * d_k))
    if out is None:
        out = torch.empty((B, T, H, d_v), dtype=q.dtype, device=q.device)
    if S_final is None and want_final:
        S_final = torch.empty((n_seq, H, d_v, d_k), dtype=torch.float32, device=q.device)
    ws_bytes = fwd_gdn2_workspace_size(B, T, H, d_k, d_v, chunk, n_seq, cu_seqlens is not None,
                                       dtype, gate, path)
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    ws_avail = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(dev, ("workspace", workspace, None, 0))
    st = _call_on(dev, lambda: lib().gdr_fwd_gdn2(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), _ptr(S0), _ptr(out), _ptr(S_final),
        B, T, H, d_k, d_v, chunk, _ptr(cu_seqlens), n_seq, dtype, gate, PATHS[path],
        _ptr(workspace), ws_avail, _stream(stream, dev)))
    if st != GDR_OK:
        raise GdrError(st, "gdr_fwd_gdn2")
    return out, S_final


def gdr_decode_step_gdn2(q, k, v, g, b, w, S, *, out=None, stream=None) -> torch.Tensor:
    """Gated DeltaNet-2 decode of one token per sequence, updating ``S`` in place."""
    N, H, d_k = q.shape
    d_v = v.shape[-1]
    dtype = _dtype_code(q)
    gate = GDR_GATE_PER_KEY_CHANNEL if g.dim() == 3 else GDR_GATE_SCALAR
    _need_contig(q, k, v, g, b, w, S)
    dev, nh = _on_cuda(q), N * H
    _check(dev, ("k", k, q.dtype, nh * d_k), ("v", v, q.dtype, nh * d_v),
           ("g", g, torch.float32, nh * (d_k if gate else 1)), ("b", b, torch.float32, nh * d_k),
           ("w", w, torch.float32, nh * d_v), ("S", S, torch.float32, nh * d_v * d_k),
           ("out", out, q.dtype, nh * d_v))
    if out is None:
        out = torch.empty((N, H, d_v), dtype=q.dtype, device=q.device)
    st = _call_on(dev, lambda: lib().gdr_decode_step_gdn2(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), _ptr(S), _ptr(out), N, H, d_k, d_v,
        dtype, gate, _stream(stream, dev)))
    if st != GDR_OK:
        raise GdrError(st, "gdr_decode_step_gdn2")
    return out


def fwd_frame_workspace_size(B, T, H, d_k, d_v, n) -> int:
    return int(lib().gdr_fwd_frame_workspace_size(B, T, H, d_k, d_v, n))


def gdr_fwd_frame(q, k, v, g, gamma, n: int, S0=None, *, out=None, S_final=None,
                  want_final: bool = True, workspace=None,
                  stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Implicit frame-level update: frames of n tokens, gamma [B,T,H], g per
    frame [B,F,H] or [B,F,H,d_k]; returns (out [B,T,H,d_v], S_final [B,H,d_v,d_k])."""
    B, T, H, d_k = q.shape
    d_v = v.shape[-1]
    dtype = _dtype_code(q)
    gate = GDR_GATE_PER_KEY_CHANNEL if g.dim() == 4 else GDR_GATE_SCALAR
    _need_contig(q, k, v, g, gamma, S0)
    dev, th, F = _on_cuda(q), B * T * H, (T + n - 1) // max(n, 1)
    _check(dev, ("k", k, q.dtype, th * d_k), ("v", v, q.dtype, th * d_v),
           ("g", g, torch.float32, B * F * H * (d_k if gate else 1)),
           ("gamma", gamma, torch.float32, th), ("S0", S0, torch.float32, B * H * d_v * d_k),
           ("out", out, q.dtype, th * d_v), ("S_final", S_final, torch.float32, B * H * d_v * d_k))
    if out is None:
        out = torch.empty((B, T, H, d_v), dtype=q.dtype, device=q.device)
    if S_final is None and want_final:
        S_final = torch.empty((B, H, d_v, d_k), dtype=torch.float32, device=q.device)
    ws_bytes = fwd_frame_workspace_size(B, max(T, 1), H, d_k, d_v, n)
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    ws_avail = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(dev, ("workspace", workspace, None, 0))
    st = _call_on(dev, lambda: lib().gdr_fwd_frame(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(gamma), _ptr(S0), _ptr(out), _ptr(S_final), B, T,
        H, d_k, d_v, n, dtype, gate, _ptr(workspace), ws_avail, _stream(stream, dev)))
    if st != GDR_OK:
        raise GdrError(st, "gdr_fwd_frame")
    return out, S_final


def gdr_decode_step(q, k, v, g, beta, S, *, out=None, stream=None) -> torch.Tensor:
    """Decode one token per sequence, updating ``S`` in place; returns out [N,H,d_v]."""
    N, H, d_k = q.shape
    d_v = v.shape[-1]
    dtype = _dtype_code(q)
    gate = GDR_GATE_PER_KEY_CHANNEL if g.dim() == 3 else GDR_GATE_SCALAR
    _need_contig(q, k, v, g, beta, S)
    dev, nh = _on_cuda(q), N * H
    _check(dev, ("k", k, q.dtype, nh * d_k), ("v", v, q.dtype, nh * d_v),
           ("g", g, torch.float32, nh * (d_k if gate else 1)), ("beta", beta, torch.float32, nh),
           ("S", S, torch.float32, nh * d_v * d_k), ("out", out, q.dtype, nh * d_v))
    if out is None:
        out = torch.empty((N, H, d_v), dtype=q.dtype, device=q.device)
    st = _call_on(dev, lambda: lib().gdr_decode_step(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), _ptr(out), N, H, d_k, d_v, dtype,
        gate, _stream(stream, dev)))
    if st != GDR_OK:
        raise GdrError(st, "gdr_decode_step")
    return out


@functools.lru_cache(maxsize=1024)
def fwd_linear_workspace_size(B, T, H, H_k, d_k, d_v, n_seq, varlen, dtype, gate,
                              path="auto") -> int:
    return int(lib().gdr_fwd_linear_workspace_size(B, T, H, H_k, d_k, d_v, n_seq,
                                                   int(bool(varlen)), dtype, gate, PATHS[path]))


@functools.lru_cache(maxsize=1024)
def bwd_linear_workspace_size(B, T, H, H_k, d_k, d_v, n_seq, varlen, dtype, gate,
                              path="auto") -> int:
    return int(lib().gdr_bwd_linear_workspace_size(B, T, H, H_k, d_k, d_v, n_seq,
                                                   int(bool(varlen)), dtype, gate, PATHS[path]))


def _linear_bad(dev, name, t, dtype, shape):
    """Raise for a tensor that _linear_args does not take."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}; expected {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    raise ValueError("tensors must be contiguous")


def _linear_refuse(q, k, v, g):
    """The reason why _linear_args does not take q, k, v, g, if there is one."""
    if not (isinstance(q, torch.Tensor) and q.is_cuda):
        raise ValueError("tensors must be CUDA tensors")
    for name, t in (("v", v), ("g", g)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    dev, lead, H, d_v = q.device, q.shape[:-2], v.shape[-2], v.shape[-1]
    if g.dim() == len(lead) + 2:
        raise ValueError("linear attention takes one decay per head ([..., H] or [H]), "
                         "not one per key channel")
    for name, t, dtype, shape in (("q", q, q.dtype, q.shape), ("k", k, q.dtype, q.shape),
                                  ("v", v, q.dtype, (*lead, H, d_v)),
                                  ("g", g, torch.float32, (H,) if g.dim() == 1 else (*lead, H))):
        if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype and
                t.is_contiguous() and t.device == dev):
            _linear_bad(dev, name, t, dtype, shape)


def _linear_rank(axes, **tensors):
    """Raise for tensors that do not have the ``axes`` of the call.  (Checked before anything is
    read from a shape: tensors of another rank can agree with each other, and the counts taken
    from their axes would then not be those of their memory.)"""
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != axes:
            raise ValueError(f"{name} has {t.dim()} axes; expected {axes}")


def _linear_args(q, k, v, g, tensors):
    """Shapes and checks shared by the linear attention calls: q, k
    [*lead, H_k, d_k], v [*lead, H, d_v], g [*lead, H] or [H]; ``tensors`` are
    further ``(name, tensor, dtype, shape)``.  Every shape must match, every
    tensor be contiguous and on q's device.  (A call for one token takes the
    host longer than the GPU, so everything is tested in one expression and the
    message made afterwards.)"""
    try:
        at, qs, vs, gs, tok, f32 = q.get_device(), q.shape, v.shape, g.shape, q.dtype, torch.float32
        good = (at >= 0 and k.shape == qs and len(vs) == len(qs) and vs[:-2] == qs[:-2] and
                (gs == vs[:-1] or len(gs) == 1 and gs[0] == vs[-2]) and
                k.dtype is tok and v.dtype is tok and g.dtype is f32 and
                k.get_device() == at and v.get_device() == at and g.get_device() == at and
                q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and g.is_contiguous())
    except AttributeError:  # not tensors
        good = False
    if not good:
        _linear_refuse(q, k, v, g)
        raise ValueError("q, k, v and g do not match")
    dev = q.device
    for spec in tensors:
        t = spec[1]
        if t is not None and not (isinstance(t, torch.Tensor) and t.shape == spec[3] and
                                  t.dtype is spec[2] and t.is_contiguous() and t.get_device() == at):
            _linear_bad(dev, *spec)
    H_k, d_k, H, d_v = qs[-2], qs[-1], vs[-2], vs[-1]
    if H_k < 1 or H % H_k:
        raise ValueError(f"{H} value heads do not share {H_k} query/key heads evenly")
    code = GDR_BF16 if tok is torch.bfloat16 else _dtype_code(q)
    return dev, code, GDR_GATE_HEAD if len(gs) == 1 else GDR_GATE_SCALAR, H, H_k, d_k, d_v


def _addr(t):
    return None if t is None else t.data_ptr()


def _linear_call(dev, stream, ws_bytes, workspace, call):
    """Run ``call(workspace address, bytes, stream handle)`` with ``dev`` current
    and, where ``stream`` is given, that stream current too: what the call
    allocates belongs to the stream that the kernels run on, so that the
    allocator hands it to no other stream while they run."""
    if workspace is not None:
        _check(dev, ("workspace", workspace, None, 0))
        _need_contig(workspace)

    def go(handle):
        ws, n = workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()
        if n < ws_bytes:
            ws, n = torch.empty(ws_bytes, dtype=torch.uint8, device=dev), ws_bytes
        return call(_addr(ws), n, handle)

    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev.index)
        if torch.cuda.current_device() == dev.index:
            return go(handle)
        with torch.cuda.device(dev):
            return go(handle)
    handle = _stream(stream, dev).value or 0
    s = stream if isinstance(stream, torch.cuda.Stream) else \
        torch.cuda.ExternalStream(handle, device=dev)
    with torch.cuda.device(dev), torch.cuda.stream(s):
        return go(handle)


def _linear_cu(cu_seqlens, B):
    if cu_seqlens is None:
        return B, 0
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be [n_seq + 1]")
    if B != 1:
        raise ValueError("a packed batch has B = 1")
    return cu_seqlens.numel() - 1, 1


def gdr_fwd_linear(q, k, v, g, S0=None, *, cu_seqlens=None, out=None, S_final=None,
                   want_final: bool = True, path: str = "auto", workspace=None,
                   stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with a decay for each head, whole sequences: q, k
    [B,T,H_k,d_k], v [B,T,H,d_v] (value heads share query/key heads when
    H_k < H), g [B,T,H] or [H]; returns ``(out [B,T,H,d_v], S_final
    [N,H,d_v,d_k] or None)``.

    bf16 tokens run on the tensor cores, where the weights of a chunk's pairs
    and the state are rounded to bf16 as operands of ``out`` (relative error of
    out 0.0023, of which its own rounding makes 0.0017; S_final keeps fp32
    accuracy); ``path="simt"`` rounds out alone, at six to sixteen times the time.

    Like every call of this module it works on the tensors' memory: results do
    not require gradients, whatever the inputs do.  For training call it and
    gdr_bwd_linear from the two sides of a ``torch.autograd.Function``."""
    if q.ndim != 4 or v.ndim != 4:
        _linear_rank(4, q=q, v=v)
    B, T = q.shape[:2]
    n_seq, varlen = _linear_cu(cu_seqlens, B)
    st_shape = (n_seq, v.shape[-2], v.shape[-1], q.shape[-1])
    dev, dtype, gate, H, H_k, d_k, d_v = _linear_args(q, k, v, g, (
        ("S0", S0, torch.float32, st_shape), ("out", out, q.dtype, v.shape),
        ("S_final", S_final, torch.float32, st_shape),
        ("cu_seqlens", cu_seqlens, torch.int32, (n_seq + 1,))))
    need = fwd_linear_workspace_size(B, T, H, H_k, d_k, d_v, n_seq, varlen, dtype, gate, path)

    def call(ws, n, handle):
        o = torch.empty_like(v) if out is None else out
        sf = S_final
        if sf is None and want_final:
            sf = torch.empty(st_shape, dtype=torch.float32, device=dev)
        return o, sf, lib().gdr_fwd_linear(
            q.data_ptr(), _addr(k), v.data_ptr(), g.data_ptr(), _addr(S0), o.data_ptr(), _addr(sf),
            B, T, H, H_k, d_k, d_v, _addr(cu_seqlens), n_seq, dtype, gate, PATHS[path], ws, n, handle)

    out, S_final, st = _linear_call(dev, stream, need, workspace, call)
    if st != GDR_OK:
        raise GdrError(st, "gdr_fwd_linear")
    return out, S_final


def gdr_decode_step_linear(q, k, v, g, S, *, out=None, stream=None) -> torch.Tensor:
    """Linear attention decode of one token per sequence, updating ``S``
    [N,H,d_v,d_k] in place: q, k [N,H_k,d_k], v [N,H,d_v], g [N,H] or [H];
    returns out [N,H,d_v]."""
    if q.ndim != 3 or v.ndim != 3:
        _linear_rank(3, q=q, v=v)
    N = q.shape[0]
    dev, dtype, gate, H, H_k, d_k, d_v = _linear_args(q, k, v, g, (
        ("S", S, torch.float32, (N, v.shape[-2], v.shape[-1], q.shape[-1])),
        ("out", out, q.dtype, v.shape)))

    def call(ws, n, handle):
        o = torch.empty_like(v) if out is None else out
        return o, lib().gdr_decode_step_linear(
            q.data_ptr(), _addr(k), v.data_ptr(), g.data_ptr(), _addr(S), o.data_ptr(), N, H,
            H_k, d_k, d_v, dtype, gate, handle)

    if stream is None and torch.cuda.current_device() == dev.index:
        out, st = call(0, 0, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        out, st = _linear_call(dev, stream, 0, None, call)
    if st != GDR_OK:
        raise GdrError(st, "gdr_decode_step_linear")
    return out


def gdr_bwd_linear(q, k, v, g, dout, S0=None, dS_final=None, *, cu_seqlens=None, dq=None, dk=None,
                   dv=None, dg=None, dS0=None, want_dS0: bool = True, path: str = "auto",
                   workspace=None, stream=None):
    """Gradients of gdr_fwd_linear from ``dout`` [B,T,H,d_v] and ``dS_final``
    [N,H,d_v,d_k] (None: zero); returns ``(dq, dk, dv, dg, dS0 or None)``,
    dq, dk and dv of the tokens' type, dg and dS0 fp32.  It takes the forward's
    inputs as they were (keep S0 where S_final was written over it) and nothing
    of its results."""
    if q.ndim != 4 or v.ndim != 4:
        _linear_rank(4, q=q, v=v)
    B, T = q.shape[:2]
    n_seq, varlen = _linear_cu(cu_seqlens, B)
    st_shape = (n_seq, v.shape[-2], v.shape[-1], q.shape[-1])
    f32 = torch.float32
    dev, dtype, gate, H, H_k, d_k, d_v = _linear_args(q, k, v, g, (
        ("dout", dout, q.dtype, v.shape), ("S0", S0, f32, st_shape),
        ("dS_final", dS_final, f32, st_shape), ("dq", dq, q.dtype, q.shape),
        ("dk", dk, q.dtype, q.shape), ("dv", dv, q.dtype, v.shape), ("dg", dg, f32, g.shape),
        ("dS0", dS0, f32, st_shape), ("cu_seqlens", cu_seqlens, torch.int32, (n_seq + 1,))))
    need = bwd_linear_workspace_size(B, T, H, H_k, d_k, d_v, n_seq, varlen, dtype, gate, path)

    def call(ws, n, handle):
        made = (torch.empty_like(q) if dq is None else dq, torch.empty_like(q) if dk is None else dk,
                torch.empty_like(v) if dv is None else dv, torch.empty_like(g) if dg is None else dg,
                torch.empty(st_shape, dtype=f32, device=dev) if dS0 is None and want_dS0 else dS0)
        return made, lib().gdr_bwd_linear(
            q.data_ptr(), _addr(k), v.data_ptr(), g.data_ptr(), _addr(S0), _addr(dout),
            _addr(dS_final), *(_addr(t) for t in made), B, T, H, H_k, d_k, d_v, _addr(cu_seqlens),
            n_seq, dtype, gate, PATHS[path], ws, n, handle)

    made, st = _linear_call(dev, stream, need, workspace, call)
    if st != GDR_OK:
        raise GdrError(st, "gdr_bwd_linear")
    return made


def device_status(stream=None) -> int:
    return int(lib().gdr_device_status(_stream(stream)))


def selftest_wait_timeout(spin_limit: int, stream=None) -> int:
    return int(lib().gdr_selftest_wait_timeout(spin_limit, _stream(stream)))


def checked_build() -> bool:
    """True when the loaded library is the checked build (gdr.h, gdr_checked_build)."""
    return bool(lib().gdr_checked_build())


def selftest_bounds(stream=None) -> int:
    return int(lib().gdr_selftest_bounds(_stream(stream)))


def set_gram_spread_limit(limit: float) -> float:
    """Set the tensor-core prefill's Gram range limit (gdr.h,
    gdr_set_gram_spread_limit); returns the previous one."""
    return float(lib().gdr_set_gram_spread_limit(float(limit)))


def profile_enable(on: bool = True) -> None:
    lib().gdr_profile_enable(1 if on else 0)


def profile_read() -> dict:
    """{kernel: (launches, total_ms)} since the previous read (then reset)."""
    res = {}
    for name, kid in KERNELS.items():
        n = ctypes.c_longlong(0)
        ms = ctypes.c_double(0.0)
        st = lib().gdr_profile_read(kid, ctypes.byref(n), ctypes.byref(ms))
        if st != GDR_OK:
            raise GdrError(st, "gdr_profile_read")
        res[name] = (int(n.value), float(ms.value))
    return res
