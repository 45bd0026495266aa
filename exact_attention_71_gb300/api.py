"""ctypes binding of libattn_sm103.so (argument marshalling only).

Every step of the attention path runs in the library's CUDA kernels; torch
is used here for device memory, streams and the tensor objects that carry
the pointers.  There is no fallback: if the library is missing or cannot be
loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libattn_sm103.so")

MODE_BLOCK, MODE_BLOCK_HADAMARD, MODE_PER_TENSOR = 0, 1, 2
BLOCK_ROWS = 128

_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    """A call into the attention library returned an error status."""

    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed ({code}): {msg}")
        self.code = code


def library() -> ctypes.CDLL:
    """Load the shared library (built by ``exact_attention_71_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m exact_attention_71_gb300.build` (needs nvcc)")
        L = ctypes.CDLL(LIB_PATH)
        P, i, f, u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_ulonglong
        L.attn_fwd.argtypes = [P, P, P, P, P, i, i, i, i, i, f, i, P]
        L.attn_fwd.restype = i
        L.attn_fwd_fp8.argtypes = [P, P, P, P, P, i, i, i, i, i, f, i, P, P, P, P]
        L.attn_fwd_fp8.restype = i
        L.attn_fwd_gqa.argtypes = [P, P, P, P, P, i, i, i, i, i, i, f, i, P]
        L.attn_fwd_gqa.restype = i
        L.attn_fwd_fp8_gqa.argtypes = [P, P, P, P, P, i, i, i, i, i, i, f, i, P, P, P, P]
        L.attn_fwd_fp8_gqa.restype = i
        L.attn_fp8_prep.argtypes = [P, P, P, i, i, i, i, i, i, u64, i, P]
        L.attn_fp8_prep_qkv.argtypes = [P, P, P, P, P, P, P, P, P, i, i, i, i, i, i, u64, P]
        L.attn_fp8_prep_qkv.restype = i
        L.attn_fp8_prep_rope.argtypes = [P, P, P, P, P, i, i, i, i, i, i, u64, i, P]
        L.attn_fp8_prep_rope.restype = i
        L.attn_fp8_prep.restype = i
        L.attn_fwd_sparse.argtypes = [P, P, P, P, P, P, i, i, i, i, i, i, f, i, P]
        L.attn_fwd_sparse.restype = i
        sz = ctypes.c_size_t
        L.attn_bwd_workspace_size.argtypes = [i, i, i, i]
        L.attn_bwd_workspace_size.restype = sz
        L.attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, sz, i, i, i, i, i, i, f, i, P]
        L.attn_bwd.restype = i
        L.attn_bwd_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, i, i, i, i, i, i, f, i, P]
        L.attn_bwd_noalloc.restype = i
        L.attn_bwd_noalloc_max_scratch.argtypes = []
        L.attn_bwd_noalloc_max_scratch.restype = sz
        L.attn_fwd_host_workspace_size.argtypes = [i, i, i, i, i]
        L.attn_fwd_host_workspace_size.restype = sz
        L.attn_fwd_host.argtypes = [P, P, P, P, P, i, i, i, i, i, i, f, i, P, sz, P]
        L.attn_fwd_host.restype = i
        L.attn_fwd_fp8_host_workspace_size.argtypes = [i, i, i, i, i]
        L.attn_fwd_fp8_host_workspace_size.restype = sz
        L.attn_fwd_fp8_host.argtypes = [P, P, P, P, P, i, i, i, i, i, i, f, i, i, u64, P, sz, P]
        L.attn_fwd_fp8_host.restype = i
        L.attn_bwd_host_workspace_size.argtypes = [i, i, i, i, i]
        L.attn_bwd_host_workspace_size.restype = sz
        L.attn_bwd_host.argtypes = [P, P, P, P, P, P, P, P, P, i, i, i, i, i, i, f, i, P, sz, P]
        L.attn_bwd_host.restype = i
        L.attn_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_int)]
        L.attn_device_status.restype = i
        L.attn_set_wait_limit.argtypes = [u64]
        L.attn_set_wait_limit.restype = i
        L.attn_last_error_string.argtypes = []
        L.attn_last_error_string.restype = ctypes.c_char_p
        L.attn_fwd_work_order.argtypes = [i, i, i, P, i]
        L.attn_fwd_work_order.restype = i
        i64 = ctypes.c_longlong
        L.attn_kv_write.argtypes = [P, P, i64, i64, P, P, P, P, P, i, i, i, i, i, i, P]
        L.attn_kv_write.restype = i
        L.attn_kv_read.argtypes = [P, P, P, P, P, i64, i, P, P, P, i, i, i, i, i, i, i, P]
        L.attn_kv_read.restype = i
        L.attn_fwd_paged_workspace_size.argtypes = [i, i, i, i, i, i, i, i]
        L.attn_fwd_paged_workspace_size.restype = sz
        L.attn_fwd_paged_plan.argtypes = [i, i, i, i, i, i, i, i, P, i]
        L.attn_fwd_paged_plan.restype = i
        L.attn_fwd_paged.argtypes = [P, P, P, P, P, P, i, P, i64, i, P, P, P, i, i, i, i, i, i, i, i, i, f, P, sz, P]
        L.attn_fwd_paged.restype = i
        _lib = L
        return _lib


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        msg = library().attn_last_error_string().decode(errors="replace")
        raise AttnError(fn, rc, msg)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _torch_stream(stream, device):
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device)


def _hold_until_done(t, stream):
    """A workspace allocated here is still in use after this function
    returns, by work on `stream` or (host-buffer entries) on the library's
    own streams, which `stream` waits for; recording the tensor on `stream`
    keeps torch's caching allocator from handing the memory out again before
    that work is done."""
    t.record_stream(_torch_stream(stream, t.device))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _check_qkv(q, k, v, dtype):
    if not (q.is_cuda and k.is_cuda and v.is_cuda):
        raise ValueError("q, k, v must be CUDA tensors")
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape:
        raise ValueError("q must be (B, N, H, d) and k, v one (B, N, H_kv, d) shape")
    B, N, H, d = q.shape
    if k.shape[0] != B or k.shape[1] != N or k.shape[3] != d or H % k.shape[2] != 0:
        raise ValueError("k, v must be (B, N, H_kv, d) with H_kv dividing the query heads")
    for t in (q, k, v):
        if t.dtype != dtype:
            raise ValueError(f"expected dtype {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous")


def _outputs(q, out, lse):
    B, N, H, d = q.shape
    if out is None:
        out = torch.empty((B, N, H, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if out.shape != (B, N, H, d) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 (B, N, H, d) tensor")
    if lse.shape != (B, H, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, H, N) tensor")
    return out, lse


def attn_fwd(q, k, v, causal: bool = False, scale: float | None = None, window: int = 0,
             out=None, lse=None, stream=None):
    """bf16 fused attention forward.  q: (B, N, H, d); k, v: (B, N, H_kv, d)
    bf16 CUDA tensors, H_kv dividing H (H_kv < H: grouped-query attention).

    Returns (O (B, N, H, d) bf16, LSE (B, H, N) float32, natural log).
    """
    _check_qkv(q, k, v, torch.bfloat16)
    out, lse = _outputs(q, out, lse)
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    if Hkv == H:
        rc = library().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d, int(bool(causal)),
                                float(scale or 0.0), int(window), ctypes.c_void_p(_stream(stream)))
        _check("attn_fwd", rc)
    else:
        rc = library().attn_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv, N, d,
                                    int(bool(causal)), float(scale or 0.0), int(window),
                                    ctypes.c_void_p(_stream(stream)))
        _check("attn_fwd_gqa", rc)
    return out, lse


def fwd_host_workspace_bytes(B: int, H: int, H_kv: int, N: int, d: int) -> int:
    return int(library().attn_fwd_host_workspace_size(B, H, H_kv, N, d))


def attn_fwd_host(q, k, v, causal: bool = False, scale: float | None = None, window: int = 0,
                  out=None, lse=None, workspace=None, device=None, stream=None):
    """attn_fwd on HOST tensors: q (B, N, H, d), k, v (B, N, H_kv, d) bf16 CPU
    tensors (page-locked, e.g. ``.pin_memory()``, for overlapped copies).
    The library stages chunks of sequences through ``workspace`` (a uint8
    CUDA tensor of at least fwd_host_workspace_bytes(...) bytes, allocated
    here when omitted) on ``device``.  Returns host (O, LSE); the call is
    asynchronous on ``stream``: synchronize it before reading them.
    """
    B, N, H, Hkv, d, out, lse = _host_args(q, k, v, out, lse)
    device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    need = fwd_host_workspace_bytes(B, H, Hkv, N, d)
    own = workspace is None
    if own:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    with torch.cuda.device(workspace.device):
        rc = library().attn_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv, N, d,
                                     int(bool(causal)), float(scale or 0.0), int(window), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(),
                                     ctypes.c_void_p(_stream(stream)))
    _check("attn_fwd_host", rc)
    if own:
        _hold_until_done(workspace, stream)
    return out, lse


def fwd_fp8_host_workspace_bytes(B: int, H: int, H_kv: int, N: int, d: int) -> int:
    return int(library().attn_fwd_fp8_host_workspace_size(B, H, H_kv, N, d))


def _host_args(q, k, v, out, lse):
    for t in (q, k, v):
        if t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("q, k, v must be contiguous 4-d bf16 CPU tensors")
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    if k.shape != v.shape or k.shape[0] != B or k.shape[1] != N or k.shape[3] != d or H % Hkv != 0:
        raise ValueError("k, v must be (B, N, H_kv, d) with H_kv dividing the query heads")
    pin = q.is_pinned()
    if out is None:
        out = torch.empty((B, N, H, d), dtype=torch.bfloat16, pin_memory=pin)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, pin_memory=pin)
    if out.is_cuda or out.shape != (B, N, H, d) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 (B, N, H, d) CPU tensor")
    if lse.is_cuda or lse.shape != (B, H, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, H, N) CPU tensor")
    return B, N, H, Hkv, d, out, lse


def attn_fwd_fp8_host(q, k, v, mode: int = MODE_BLOCK_HADAMARD, sign_seed: int = 0, causal: bool = False,
                      scale: float | None = None, window: int = 0, out=None, lse=None, workspace=None, device=None,
                      stream=None):
    """The FP8 path on HOST bf16 tensors (prep + e4m3 forward per chunk of
    sequences, staged and overlapped like attn_fwd_host).  mode: MODE_BLOCK or
    MODE_BLOCK_HADAMARD.  Returns host (O, LSE); asynchronous on ``stream``."""
    B, N, H, Hkv, d, out, lse = _host_args(q, k, v, out, lse)
    device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    own = workspace is None
    if own:
        need = fwd_fp8_host_workspace_bytes(B, H, Hkv, N, d)
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    with torch.cuda.device(workspace.device):
        rc = library().attn_fwd_fp8_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv, N, d,
                                         int(bool(causal)), float(scale or 0.0), int(window), int(mode),
                                         int(sign_seed) & 0xFFFFFFFFFFFFFFFF, _ptr(workspace),
                                         workspace.numel() * workspace.element_size(),
                                         ctypes.c_void_p(_stream(stream)))
    _check("attn_fwd_fp8_host", rc)
    if own:
        _hold_until_done(workspace, stream)
    return out, lse


def attn_fwd_sparse(q, k, v, block_mask, causal: bool = False, scale: float | None = None, window: int = 0,
                    out=None, lse=None, stream=None):
    """bf16 forward with a block-sparse key mask: block_mask is a uint8 (or
    bool) CUDA tensor (B, H, T, T), T = ceil(N / 128); query block i of
    (b, h) sees key block j iff block_mask[b, h, i, j] != 0 (ANDed with the
    causal / window masks).  Rows that see no key get O = 0, LSE = -inf."""
    _check_qkv(q, k, v, torch.bfloat16)
    out, lse = _outputs(q, out, lse)
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    T = (N + 127) // 128
    if block_mask.dtype == torch.bool:
        block_mask = block_mask.to(torch.uint8)
    if (block_mask.dtype != torch.uint8 or not block_mask.is_cuda or not block_mask.is_contiguous()
            or tuple(block_mask.shape) != (B, H, T, T)):
        raise ValueError(f"block_mask must be a contiguous uint8 CUDA tensor of shape ({B}, {H}, {T}, {T})")
    rc = library().attn_fwd_sparse(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(block_mask), B, H, Hkv, N,
                                   d, int(bool(causal)), float(scale or 0.0), int(window),
                                   ctypes.c_void_p(_stream(stream)))
    _check("attn_fwd_sparse", rc)
    return out, lse


def bwd_host_workspace_bytes(B: int, H: int, H_kv: int, N: int, d: int) -> int:
    return int(library().attn_bwd_host_workspace_size(B, H, H_kv, N, d))


def attn_bwd_host(dout, q, k, v, out, lse, causal: bool = False, scale: float | None = None, window: int = 0,
                  dq=None, dk=None, dv=None, workspace=None, device=None, stream=None):
    """attn_bwd on HOST tensors (bf16 CPU q, dout, out (B, N, H, d); k, v
    (B, N, H_kv, d); float32 lse (B, H, N)), staged through ``workspace`` (at
    least bwd_host_workspace_bytes(...) bytes on ``device``) like
    attn_fwd_host.  Returns host (dq, dk, dv); asynchronous on ``stream``."""
    B, N, H, Hkv, d, _, _ = _host_args(q, k, v, out, lse)
    if dout.is_cuda or dout.shape != q.shape or dout.dtype != torch.bfloat16 or not dout.is_contiguous():
        raise ValueError("dout must be a contiguous bf16 CPU tensor shaped like q")
    pin = q.is_pinned()
    dq = torch.empty(q.shape, dtype=torch.bfloat16, pin_memory=pin) if dq is None else dq
    dk = torch.empty(k.shape, dtype=torch.bfloat16, pin_memory=pin) if dk is None else dk
    dv = torch.empty(v.shape, dtype=torch.bfloat16, pin_memory=pin) if dv is None else dv
    for t, ref in ((dq, q), (dk, k), (dv, v)):
        if t.is_cuda or t.shape != ref.shape or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("dq, dk, dv must be contiguous bf16 CPU tensors shaped like q, k, v")
    device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    own = workspace is None
    if own:
        workspace = torch.empty(max(bwd_host_workspace_bytes(B, H, Hkv, N, d), 256), dtype=torch.uint8,
                                device=device)
    with torch.cuda.device(workspace.device):
        rc = library().attn_bwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq),
                                     _ptr(dk), _ptr(dv), B, H, Hkv, N, d, int(bool(causal)), float(scale or 0.0),
                                     int(window), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     ctypes.c_void_p(_stream(stream)))
    _check("attn_bwd_host", rc)
    if own:
        _hold_until_done(workspace, stream)
    return dq, dk, dv


def bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(library().attn_bwd_workspace_size(B, H, N, d))


def attn_bwd(dout, q, k, v, out, lse, causal: bool = False, scale: float | None = None, window: int = 0,
             dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward of attn_fwd: (dq, dk, dv) for the upstream gradient dout.

    q, dout, out: bf16 (B, N, H, d); k, v: bf16 (B, N, H_kv, d); lse: the
    forward's float32 (B, H, N).  workspace: optional uint8 CUDA tensor of at
    least bwd_workspace_bytes(B, H, N, d) bytes (allocated per call when
    omitted).
    """
    _check_qkv(q, k, v, torch.bfloat16)
    for t, name in ((dout, "dout"), (out, "out")):
        if t.shape != q.shape or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.device != q.device:
            raise ValueError(f"{name} must be a contiguous bf16 tensor shaped like q")
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    if lse.shape != (B, H, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, H, N) tensor")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = bwd_workspace_bytes(B, H, N, d)
    own = workspace is None
    if own:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    rc = library().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                            _ptr(dv), _ptr(workspace), workspace.numel() * workspace.element_size(), B, H, Hkv, N, d,
                            int(bool(causal)), float(scale or 0.0), int(window), ctypes.c_void_p(_stream(stream)))
    _check("attn_bwd", rc)
    if own and stream is not None:
        _hold_until_done(workspace, stream)   # the launches run on `stream`, not torch's current one
    return dq, dk, dv


def attn_bwd_noalloc(dout, q, k, v, out, lse, causal: bool = False, scale: float | None = None, window: int = 0,
                     dq=None, dk=None, dv=None, stream=None):
    """attn_bwd without a workspace: the library's built-in device scratch
    buffer is used instead (for callers that may not allocate; calls on one
    device must not overlap on the GPU).  dq, dk, dv are allocated here only
    when not given."""
    _check_qkv(q, k, v, torch.bfloat16)
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    rc = library().attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq),
                                    _ptr(dk), _ptr(dv), B, H, Hkv, N, d, int(bool(causal)), float(scale or 0.0),
                                    int(window), ctypes.c_void_p(_stream(stream)))
    _check("attn_bwd_noalloc", rc)
    return dq, dk, dv


def attn_fp8_prep(x, mode: int = MODE_BLOCK_HADAMARD, sign_seed: int = 0, is_v: bool = False,
                  out=None, scales=None, stream=None):
    """Rotation (mode 1, not V) + block quantisation of one bf16 (B,N,H,d) tensor.

    Returns (codes as a torch.uint8 (B,N,H,d) tensor, scales float32 (B,H,ceil(N/128))).
    """
    if not x.is_cuda or x.dtype != torch.bfloat16 or x.dim() != 4 or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 (B, N, H, d) CUDA tensor")
    B, N, H, d = x.shape
    nblk = (N + BLOCK_ROWS - 1) // BLOCK_ROWS
    if out is None:
        out = torch.empty((B, N, H, d), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((B, H, nblk), dtype=torch.float32, device=x.device)
    rc = library().attn_fp8_prep(_ptr(x), _ptr(out), _ptr(scales), B, H, N, d, BLOCK_ROWS, int(mode),
                                 int(sign_seed) & 0xFFFFFFFFFFFFFFFF, int(bool(is_v)),
                                 ctypes.c_void_p(_stream(stream)))
    _check("attn_fp8_prep", rc)
    return out, scales


def attn_fwd_fp8(q8, k8, v8, q_scale, k_scale, v_scale, causal: bool = False, scale: float | None = None,
                 window: int = 0, out=None, lse=None, stream=None):
    """FP8 e4m3 fused attention forward on codes from attn_fp8_prep.

    q8, k8, v8: uint8 (or float8_e4m3fn) (B, N, H, d) CUDA tensors; *_scale:
    float32 (B, H, ceil(N/128)).  Returns (O bf16 (B,N,H,d), LSE (B,H,N)).
    """
    for t in (q8, k8, v8):
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q8, k8, v8 must be contiguous e4m3 codes on the GPU")
    if q8.dim() != 4 or k8.dim() != 4 or k8.shape != v8.shape:
        raise ValueError("q8 must be (B, N, H, d) and k8, v8 one (B, N, H_kv, d) shape")
    B, N, H, d = q8.shape
    Hkv = k8.shape[2]
    if k8.shape[0] != B or k8.shape[1] != N or k8.shape[3] != d or H % Hkv != 0:
        raise ValueError("k8, v8 must be (B, N, H_kv, d) with H_kv dividing the query heads")
    nblk = (N + BLOCK_ROWS - 1) // BLOCK_ROWS
    for s, heads in ((q_scale, H), (k_scale, Hkv), (v_scale, Hkv)):
        if s.shape != (B, heads, nblk) or s.dtype != torch.float32 or not s.is_contiguous():
            raise ValueError("scales must be contiguous float32 (B, heads, ceil(N/128)) tensors")
    out, lse = _outputs(q8, out, lse)
    rc = library().attn_fwd_fp8_gqa(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(out), _ptr(lse), B, H, Hkv, N, d,
                                    int(bool(causal)), float(scale or 0.0), int(window), _ptr(q_scale),
                                    _ptr(k_scale), _ptr(v_scale), ctypes.c_void_p(_stream(stream)))
    _check("attn_fwd_fp8_gqa", rc)
    return out, lse


def attn_fp8_prep_rope(x, rope_cos, rope_sin, mode: int = MODE_BLOCK_HADAMARD, sign_seed: int = 0,
                       interleaved: bool = False, out=None, scales=None, stream=None):
    """RoPE fused with the FP8 prep of Q or K: each row of token n is turned
    by the (N, d/2) float32 cos / sin tables (pairs (i, i + d/2), or (2i, 2i+1)
    when interleaved), then rotated (mode 1) and block-quantised.

    Returns (codes uint8 (B,N,H,d), scales float32 (B,H,ceil(N/128))).
    """
    if not x.is_cuda or x.dtype != torch.bfloat16 or x.dim() != 4 or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 (B, N, H, d) CUDA tensor")
    B, N, H, d = x.shape
    for t in (rope_cos, rope_sin):
        if (not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous() or t.shape != (N, d // 2)
                or t.device != x.device):
            raise ValueError("rope_cos / rope_sin must be contiguous float32 (N, d/2) tensors on x's device")
    nblk = (N + BLOCK_ROWS - 1) // BLOCK_ROWS
    if out is None:
        out = torch.empty((B, N, H, d), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((B, H, nblk), dtype=torch.float32, device=x.device)
    rc = library().attn_fp8_prep_rope(_ptr(x), _ptr(out), _ptr(scales), _ptr(rope_cos), _ptr(rope_sin),
                                      B, H, N, d, BLOCK_ROWS, int(mode), int(sign_seed) & 0xFFFFFFFFFFFFFFFF,
                                      int(bool(interleaved)), ctypes.c_void_p(_stream(stream)))
    _check("attn_fp8_prep_rope", rc)
    return out, scales


def attn_fp8_prep_qkv(q, k, v, mode: int = MODE_BLOCK_HADAMARD, sign_seed: int = 0, stream=None):
    """The prep of Q, K (rotated in mode 1) and V (never rotated) in one call
    (one launch for modes 0 and 1 at head dims 64 and 128).

    Returns (q8, k8, v8, q_scale, k_scale, v_scale)."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 (B, N, H, d) CUDA tensor")
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, N, Hkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be (B, N, H_kv, d) with q's B, N and d")
    nblk = (N + BLOCK_ROWS - 1) // BLOCK_ROWS
    q8 = torch.empty((B, N, H, d), dtype=torch.uint8, device=q.device)
    k8 = torch.empty((B, N, Hkv, d), dtype=torch.uint8, device=q.device)
    v8 = torch.empty((B, N, Hkv, d), dtype=torch.uint8, device=q.device)
    qs = torch.empty((B, H, nblk), dtype=torch.float32, device=q.device)
    ks = torch.empty((B, Hkv, nblk), dtype=torch.float32, device=q.device)
    vs = torch.empty((B, Hkv, nblk), dtype=torch.float32, device=q.device)
    rc = library().attn_fp8_prep_qkv(_ptr(q), _ptr(k), _ptr(v), _ptr(q8), _ptr(k8), _ptr(v8), _ptr(qs), _ptr(ks),
                                     _ptr(vs), B, H, Hkv, N, d, int(mode), int(sign_seed) & 0xFFFFFFFFFFFFFFFF,
                                     ctypes.c_void_p(_stream(stream)))
    _check("attn_fp8_prep_qkv", rc)
    return q8, k8, v8, qs, ks, vs


def fp8_prepare_qkv(q, k, v, mode: int = MODE_BLOCK_HADAMARD, sign_seed: int = 0, stream=None, rope=None):
    """Runs the prep on Q, K (rotated in mode 1) and V (never rotated), one
    launch where the library has it (attn_fp8_prep_qkv).
    rope: optional (cos, sin, interleaved); RoPE is then fused into the prep
    of Q and K."""
    if rope is None:
        return attn_fp8_prep_qkv(q, k, v, mode, sign_seed, stream=stream)
    else:
        c, s_, il = rope
        q8, qs = attn_fp8_prep_rope(q, c, s_, mode, sign_seed, il, stream=stream)
        k8, ks = attn_fp8_prep_rope(k, c, s_, mode, sign_seed, il, stream=stream)
    v8, vs = attn_fp8_prep(v, mode, sign_seed, True, stream=stream)
    return q8, k8, v8, qs, ks, vs


CACHE_BF16, CACHE_E4M3 = 0, 1


class KVCache(NamedTuple):
    """A paged key/value cache on the GPU: k and v are (num_pages, H_kv,
    page_size, d), bf16, or e4m3 codes (uint8 or float8_e4m3fn) with the float32
    row scales (num_pages, H_kv, page_size) beside them (None for bf16)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None


def kv_cache(num_pages: int, page_size: int, H_kv: int, d: int, e4m3: bool = True, device=None) -> KVCache:
    """A KVCache of zeros on `device` (default: the current one)."""
    device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    shape = (num_pages, H_kv, page_size, d)
    dtype = torch.uint8 if e4m3 else torch.bfloat16
    k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    if not e4m3:
        return KVCache(k, v)
    ks, vs = (torch.ones(shape[:3], dtype=torch.float32, device=device) for _ in range(2))
    return KVCache(k, v, ks, vs)


# The paged entries are called once per layer and decoding step, where the host
# is the bound: one pass of checks, devices compared by their index, plain
# integers to ctypes, no context manager unless the device asks for one.

_BF16, _F32, _I32, _I64, _U8, _E4M3 = (torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8,
                                       torch.float8_e4m3fn)


def _check_cache(cache):
    """(num_pages, H_kv, page_size, d, cache dtype, device index, pointers) of a KVCache."""
    k, v, ks, vs = cache
    shape, dtype, dev = k.shape, k.dtype, k.get_device()
    if not k.is_cuda or len(shape) != 4 or v.shape != shape or v.dtype != dtype or v.get_device() != dev:
        raise ValueError("cache k and v must be CUDA tensors of one (num_pages, H_kv, page_size, d) shape and dtype")
    if not k.is_contiguous() or not v.is_contiguous():
        raise ValueError("cache k and v must be contiguous")
    pages, Hkv, ps, d = shape
    if dtype == _BF16:
        if ks is not None or vs is not None:
            raise ValueError("a bf16 cache has no scales")
        return pages, Hkv, ps, d, CACHE_BF16, dev, (k.data_ptr(), v.data_ptr(), None, None)
    if dtype != _U8 and dtype != _E4M3:
        raise ValueError("cache k and v must be bf16 or e4m3 codes (uint8 or float8_e4m3fn)")
    rows = shape[:3]
    if (ks is None or vs is None or ks.dtype != _F32 or vs.dtype != _F32 or ks.shape != rows or vs.shape != rows
            or not ks.is_contiguous() or not vs.is_contiguous() or ks.get_device() != dev or vs.get_device() != dev):
        raise ValueError("an e4m3 cache has contiguous float32 (num_pages, H_kv, page_size) scales on its device")
    return pages, Hkv, ps, d, CACHE_E4M3, dev, (k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr())


def _check_table(block_table, seq_lens, B, dev):
    """(max_pages, row stride) of a block table."""
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != B or block_table.dtype != _I32 or block_table.get_device() != dev:
        raise ValueError("block_table must be an int32 (B, max_pages) tensor with contiguous rows on the cache's device")
    max_pages = shape[1]
    stride, step = block_table.stride()
    if max_pages > 1 and step != 1:
        raise ValueError("block_table must be an int32 (B, max_pages) tensor with contiguous rows on the cache's device")
    if (seq_lens.shape != (B,) or seq_lens.dtype != _I32 or seq_lens.get_device() != dev
            or not seq_lens.is_contiguous()):
        raise ValueError("seq_lens must be a contiguous int32 (B,) tensor on the cache's device")
    if B <= 1:
        stride = max_pages
    elif stride < max_pages:
        raise ValueError("the rows of block_table must not overlap")
    return max_pages, stride


# Entries of torch that are not public and may go away or change; without them the
# public ones are called (an attention call of 19 us on the host then takes 26: the
# dispatcher's part of a torch.empty costs more than the allocation).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_empty = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_fills = torch.are_deterministic_algorithms_enabled
_watchers = [getattr(torch._C, n, None) for n in ("_len_torch_dispatch_stack", "_len_torch_function_stack")]


def _unwatched() -> bool:
    """Whether nothing is to see or fill the memory that is allocated: no dispatch or
    function mode is active, and torch fills no uninitialised memory."""
    try:
        for active in _watchers:
            if active():
                return False
    except TypeError:
        return False
    return not _fills()


def _current_raw_stream(dev: int) -> int:
    if _raw_stream is not None:
        try:
            return _raw_stream(dev)
        except TypeError:
            pass
    return torch.cuda.current_stream(dev).cuda_stream


def _launch(fn, name, dev, stream, args):
    """Calls entry `fn` with `args` and the stream, with device `dev` current."""
    raw = _current_raw_stream(dev) if stream is None else _stream(stream)
    if _current_device() == dev:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, raw)
    if rc != 0:
        _check(name, rc)


def attn_kv_write(k, v, slots, cache: KVCache, stream=None) -> None:
    """Writes the keys and values of T new tokens into their slots of the
    cache, quantising each row for an e4m3 cache (scale = amax / 448 per token
    and head).

    k, v: bf16 (T, H_kv, d) CUDA tensors; a token's heads are contiguous, tokens
    may be strided (columns of one projection).  slots: int64 (T,), page *
    page_size + row; negative slots are skipped, those >= 0 must differ.  A slot
    beyond the cache is skipped and reported by device_status().
    """
    pages, Hkv, ps, d, dtype, dev, ptrs = _check_cache(cache)
    shape = k.shape
    if len(shape) != 3 or v.shape != shape or shape[1] != Hkv or shape[2] != d:
        raise ValueError(f"k and v must be (T, {Hkv}, {d}) tensors")
    T = shape[0]
    strides = []
    for t in (k, v):
        if t.dtype != _BF16 or t.get_device() != dev:
            raise ValueError("k and v must be bf16 tensors on the cache's device")
        s0, s1, s2 = t.stride()
        if s2 != 1 or (Hkv > 1 and s1 != d):
            raise ValueError("a token's heads must be contiguous in k and v")
        strides.append(s0 if T > 1 else Hkv * d)
    if slots.shape != (T,) or slots.dtype != _I64 or slots.get_device() != dev or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous int64 (T,) tensor on the cache's device")
    _launch(library().attn_kv_write, "attn_kv_write", dev, stream,
            (k.data_ptr(), v.data_ptr(), *strides, slots.data_ptr(), *ptrs, T, Hkv, d, pages, ps, dtype))


def attn_kv_read(cache: KVCache, block_table, seq_lens, N: int, out_k=None, out_v=None, stream=None):
    """The first min(seq_lens[b], N) tokens of every sequence as bf16 (B, N,
    H_kv, d) keys and values (e4m3: scale * value, rounded once).

    block_table: int32 (B, max_pages), rows may be strided; seq_lens: int32
    (B,).  Rows from a sequence's length on are left as they were in out_k /
    out_v (zeros where these are allocated here).  Returns (k, v).
    """
    pages, Hkv, ps, d, dtype, dev, ptrs = _check_cache(cache)
    B = block_table.shape[0]
    max_pages, stride = _check_table(block_table, seq_lens, B, dev)
    shape = (B, N, Hkv, d)
    if out_k is None or out_v is None:
        # (the zeros are written on the launch's stream)
        with torch.cuda.stream(_torch_stream(stream, cache.k.device)):
            out_k = torch.zeros(shape, dtype=_BF16, device=cache.k.device) if out_k is None else out_k
            out_v = torch.zeros(shape, dtype=_BF16, device=cache.k.device) if out_v is None else out_v
    for t in (out_k, out_v):
        if t.shape != shape or t.dtype != _BF16 or not t.is_contiguous() or t.get_device() != dev:
            raise ValueError(f"out_k and out_v must be contiguous bf16 {shape} tensors on the cache's device")
    _launch(library().attn_kv_read, "attn_kv_read", dev, stream,
            (*ptrs, block_table.data_ptr(), stride, max_pages, seq_lens.data_ptr(), out_k.data_ptr(), out_v.data_ptr(),
             B, N, Hkv, d, pages, ps, dtype))
    return out_k, out_v


@functools.lru_cache(maxsize=1024)
def paged_workspace_bytes(B: int, Nq: int, H: int, H_kv: int, d: int, prefix_len: int, max_pages: int,
                          page_size: int) -> int:
    return int(library().attn_fwd_paged_workspace_size(B, Nq, H, H_kv, d, prefix_len, max_pages, page_size))


class PagedPlan(NamedTuple):
    """How attn_fwd_paged cuts up a call: the kernel ("stream", "tile" or None) of the
    prefix and of the own tokens, their key ranges, the query rows of a streaming
    CTA, the 128-row tiles of a key/value head in the tile kernel, and whether the
    one range there is is written without a join."""
    prefix_kernel: str | None
    own_kernel: str
    prefix_parts: int
    own_parts: int
    stream_rows: int
    prefix_row_tiles: int
    own_row_tiles: int
    direct: bool


def paged_plan(B: int, Nq: int, H: int, H_kv: int, d: int, prefix_len: int, max_pages: int,
               page_size: int) -> PagedPlan | None:
    """Host only: the plan of a call of these sizes; None for empty or refused ones."""
    buf = (ctypes.c_int * 8)()
    if library().attn_fwd_paged_plan(B, Nq, H, H_kv, d, prefix_len, max_pages, page_size,
                                     ctypes.cast(buf, ctypes.c_void_p), 8) != 8:
        return None
    kernels = (None, "stream", "tile")
    return PagedPlan(kernels[buf[0]], kernels[buf[1]], *buf[2:7], bool(buf[7]))


def _paged_buffers(out, lse, workspace, need, B, Nq, H, d, dev):
    """out, lse and a workspace of `need` bytes, allocated where they are None."""
    if _raw_empty is not None and _current_device() == dev and _unwatched():
        try:
            if out is None:
                out = _raw_empty((B, Nq, H, d), (Nq * H * d, H * d, d, 1), _BF16)
            if lse is None:
                lse = _raw_empty((B, H, Nq), (H * Nq, Nq, 1), _F32)
            if workspace is None and need:
                workspace = _raw_empty((need,), (1,), _U8)
            return out, lse, workspace
        except TypeError:            # (another signature: the public way, below)
            pass
    device = torch.device("cuda", dev)
    if out is None:
        out = torch.empty((B, Nq, H, d), dtype=_BF16, device=device)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=_F32, device=device)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=_U8, device=device)
    return out, lse, workspace


def attn_fwd_paged(q, cache: KVCache, block_table, seq_lens, prefix_table=None, prefix_len: int = 0,
                   causal: bool = True, scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """Attention of Nq query tokens of each of B sequences over the paged cache:
    the shared prefix (read once for the whole batch) followed by each
    sequence's own tokens, whose last Nq are the queries.

    q: bf16 (B, Nq, H, d); block_table: int32 (B, max_pages), the own pages (rows
    may be strided, e.g. a full table without its shared columns); seq_lens:
    int32 (B,), the own tokens; prefix_table: int32 (>= ceil(prefix_len /
    page_size),); prefix_len: host int.  causal: query i sees own keys j <=
    seq_lens[b] - Nq + i (all of them otherwise), and the whole prefix; there is no
    sliding window.
    workspace: optional uint8 CUDA tensor of at least paged_workspace_bytes(...)
    bytes, scratch.  out, lse and workspace that are not given are allocated on
    the launch's stream.  Returns (O (B, Nq, H, d) bf16, LSE (B, H, Nq) float32).
    """
    pages, Hkv, ps, d, dtype, dev, ptrs = _check_cache(cache)
    shape = q.shape
    if len(shape) != 4 or q.dtype != _BF16 or q.get_device() != dev or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 (B, Nq, H, d) tensor on the cache's device")
    B, Nq, H, dq = shape
    if dq != d or Hkv == 0 or H % Hkv != 0:
        raise ValueError("q's head dim must be the cache's and its heads a multiple of the cache's")
    max_pages, stride = _check_table(block_table, seq_lens, B, dev)
    prefix_len = int(prefix_len)
    prefix = None
    if prefix_len > 0:
        if (prefix_table is None or len(prefix_table.shape) != 1 or prefix_table.dtype != _I32
                or prefix_table.get_device() != dev or not prefix_table.is_contiguous()
                or prefix_table.shape[0] * ps < prefix_len):
            raise ValueError("prefix_table must be a contiguous int32 tensor of prefix_len's pages on the cache's device")
        prefix = prefix_table.data_ptr()
    if out is not None and (out.shape != shape or out.dtype != _BF16 or not out.is_contiguous()
                            or out.get_device() != dev):
        raise ValueError("out must be a contiguous bf16 (B, Nq, H, d) tensor on the cache's device")
    if lse is not None and (lse.shape != (B, H, Nq) or lse.dtype != _F32 or not lse.is_contiguous()
                            or lse.get_device() != dev):
        raise ValueError("lse must be a contiguous float32 (B, H, Nq) tensor on the cache's device")
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    need = 0
    if workspace is None:
        need = paged_workspace_bytes(B, Nq, H, Hkv, d, prefix_len, max_pages, ps)
    if stream is None:
        out, lse, workspace = _paged_buffers(out, lse, workspace, need, B, Nq, H, d, dev)
    else:
        # (memory of the launch's stream: that of another may still be in use there)
        with torch.cuda.stream(_torch_stream(stream, q.device)):
            out, lse, workspace = _paged_buffers(out, lse, workspace, need, B, Nq, H, d, dev)
    ws = None
    if workspace is not None:
        ws = workspace.data_ptr()
        if need == 0:
            need = workspace.numel() * workspace.element_size()
    _launch(library().attn_fwd_paged, "attn_fwd_paged", dev, stream,
            (q.data_ptr(), *ptrs, prefix, prefix_len, block_table.data_ptr(), stride, max_pages, seq_lens.data_ptr(),
             out.data_ptr(), lse.data_ptr(), B, Nq, H, Hkv, d, pages, ps, dtype, 1 if causal else 0,
             float(scale or 0.0), ws, need))
    return out, lse


def device_status(stream=None):
    """(status, site): waits for the stream and reads/clears the status word."""
    site = ctypes.c_int(0)
    rc = library().attn_device_status(ctypes.c_void_p(_stream(stream)), ctypes.byref(site))
    return rc, site.value


def fwd_work_order(n_mblocks: int, bh: int, grid: int):
    """The causal d=128 forward's work order (host only): a list of
    (query block, batch*head) per item, or None where the launch uses the
    closed-form order."""
    n = n_mblocks * bh
    buf = (ctypes.c_uint * max(n, 1))()
    got = library().attn_fwd_work_order(n_mblocks, bh, grid, ctypes.cast(buf, ctypes.c_void_p), n)
    if got == 0:
        return None
    return [(buf[k] & 0xFFFF, buf[k] >> 16) for k in range(got)]


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)
