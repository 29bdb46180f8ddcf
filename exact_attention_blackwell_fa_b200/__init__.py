"""Exact scaled-dot-product attention (forward and backward) for B200 / sm_100a.

Thin Python binding over the C ABI in include/fa.h (libfa.so).  PyTorch supplies
device memory and the current stream; every step of the computation runs in the
library's CUDA kernels.  The functions carry the C names:

    fa_fwd(q, k, v, causal=False, scale=None) -> (o, lse)
    fa_fwd_splitkv(q, k, v, causal=False, scale=None, num_splits=0) -> (o, lse)
    fa_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                  seqused_k=None, causal=False, scale=None) -> (o, lse)
    fa_bwd(q, k, v, o, lse, dout, causal=False, scale=None) -> (dq, dk, dv)
    fa_bwd_varlen(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                  max_seqlen_k, seqused_k=None, causal=False, scale=None) -> (dq, dk, dv)
    fa_bwd_workspace_size(B, Sq, Hq, d) -> int
    fa_bwd_noalloc(q, k, v, o, lse, dout, causal=False, scale=None) -> (dq, dk, dv)
    fa_kv_cache_size(num_pages, page_size, Hkv, d, fmt=FA_KV_16) -> int
    fa_kv_append(q, k, v, k_cache, v_cache, cu_seqlens, seqlens_k, block_table, inv_freq=None,
                 interleaved=False) -> q_out        # rotates q and k, fills the paged caches
    fa_kv_gather(k_cache, v_cache, cu_seqlens_k, block_table, total_k, dtype=None) -> (k, v)
    fa_fwd_paged(q, k_cache, v_cache, cu_seqlens_q, seqlens_k, block_table, max_seqlen_q,
                 causal=False, scale=None) -> (o, lse)
    fa_fwd_paged_workspace_size(B, max_seqlen_q, Hq, Hkv, d) -> int
    fa_status_string(code) -> str
    fa_last_device_status() -> (code, detail)
    fa_clear_device_status()
    fa_set_unit_schedule(mode)        # FA_SCHED_STATIC (0), FA_SCHED_CLC (1), FA_SCHED_AUTO (2, default)
    fa_set_exp2_emulation(pairs_of_4) # forward exp2 split: -1 default, 0..3 of 4 on the FMA pipe
    fa_set_wait_timeout_ms(ms)        # limit of a kernel's pipeline waits (default 1000)
    fa_debug_inject(mode)
    fa_debug_exp2(x, mode=0) -> y

Tensors are CUDA, contiguous, [batch, seq, heads, head_dim], bf16 or fp16; LSE is
float32 [batch, Hq, Sq].  A non-OK status raises FAError; nothing falls back.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import _lib

__all__ = [
    "FAError", "fa_fwd", "fa_fwd_splitkv", "fa_fwd_varlen", "fa_bwd", "fa_bwd_varlen", "fa_bwd_noalloc", "fa_bwd_workspace_size", "fa_status_string",
    "fa_kv_cache_size", "fa_kv_append", "fa_kv_gather", "fa_fwd_paged", "fa_fwd_paged_workspace_size", "FA_KV_16", "FA_KV_INT4",
    "fa_last_device_status", "fa_clear_device_status", "fa_set_unit_schedule", "fa_set_exp2_emulation", "fa_set_wait_timeout_ms", "fa_debug_inject", "fa_debug_exp2",
    "FA_SCHED_STATIC", "FA_SCHED_CLC", "FA_SCHED_AUTO",
]

FA_SCHED_STATIC, FA_SCHED_CLC, FA_SCHED_AUTO = 0, 1, 2
FA_KV_16, FA_KV_INT4 = _lib.FA_KV_16, _lib.FA_KV_INT4


class FAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {fa_status_string(code)}")


def fa_status_string(code: int) -> str:
    return _lib.load().fa_status_string(int(code)).decode()


def _stream_ptr(stream) -> int:
    """The stream handle to launch on: the given one, else the current device's current
    stream (the wrappers make q's device current first)."""
    if stream is None:
        if not torch.cuda.is_initialized():
            torch.cuda.init()
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t) -> int:
    dtype = t if isinstance(t, torch.dtype) else t.dtype
    if dtype == torch.bfloat16:
        return _lib.FA_BF16
    if dtype == torch.float16:
        return _lib.FA_FP16
    raise TypeError(f"fa: inputs must be bf16 or fp16, got {dtype}")


def _check(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"fa: {name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"fa: {name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"fa: {name} has dtype {t.dtype}, expected {dtype}")


def _same_device(ref: torch.Tensor, **tensors):
    """Every tensor must sit on ref's device: the library launches on the current
    device, which the wrappers set to ref's."""
    for name, t in tensors.items():
        if t is not None and t.device != ref.device:
            raise ValueError(f"fa: {name} is on {t.device}, expected {ref.device}")


def _shape(t: torch.Tensor, name: str, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"fa: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check_kv(q, k, v, packed: bool):
    if packed:
        if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape or k.shape[2] != q.shape[2]:
            raise ValueError("fa: q must be [total_q, Hq, d] and k, v [total_k, Hkv, d] with the same d")
    elif q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or k.shape[0] != q.shape[0] or \
            k.shape[3] != q.shape[3]:
        raise ValueError("fa: q must be [B, Sq, Hq, d] and k, v [B, Sk, Hkv, d] matching q")


def _workspace(ws, ref: torch.Tensor, need: int, name: str = "workspace"):
    if ws is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=ref.device)
    _check(ws, name)
    _same_device(ref, **{name: ws})
    if ws.numel() * ws.element_size() < need:
        raise ValueError(f"fa: {name} holds {ws.numel() * ws.element_size()} bytes, needs {need}")
    return ws


def _raise(code: int, where: str):
    if code != _lib.FA_OK:
        raise FAError(code, where)


def fa_fwd(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
           stream=None):
    """Forward. q [B,Sq,Hq,d], k/v [B,Sk,Hkv,d] -> (o [B,Sq,Hq,d], lse [B,Hq,Sq] fp32)."""
    _check(q, "q")
    _check(k, "k", q.dtype)
    _check(v, "v", q.dtype)
    _check_kv(q, k, v, packed=False)
    B, Sq, Hq, d = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hq, Sq, dtype=torch.float32, device=q.device)
    _check(out, "out", q.dtype)
    _check(lse, "lse", torch.float32)
    _shape(out, "out", q.shape)
    _shape(lse, "lse", (B, Hq, Sq))
    _same_device(q, k=k, v=v, out=out, lse=lse)
    with torch.cuda.device(q.device):
        code = _lib.load().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                  lse.data_ptr(), B, Sq, Sk, Hq, Hkv, d, int(bool(causal)),
                                  float(scale), _dtype_code(q), _stream_ptr(stream))
    _raise(code, "fa_fwd")
    return out, lse


def fa_fwd_splitkv(q, k, v, causal: bool = False, scale: float | None = None, num_splits: int = 0,
                   out=None, lse=None, workspace=None, stream=None):
    """Split-KV forward (decode-shaped calls): same layouts and result as fa_fwd.
    num_splits <= 0 lets the library choose."""
    _check(q, "q")
    _check(k, "k", q.dtype)
    _check(v, "v", q.dtype)
    _check_kv(q, k, v, packed=False)
    B, Sq, Hq, d = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty(B, Hq, Sq, dtype=torch.float32, device=q.device)
    _check(out, "out", q.dtype)
    _check(lse, "lse", torch.float32)
    _shape(out, "out", q.shape)
    _shape(lse, "lse", (B, Hq, Sq))
    _same_device(q, k=k, v=v, out=out, lse=lse)
    lib = _lib.load()
    with torch.cuda.device(q.device):
        need = int(lib.fa_fwd_splitkv_workspace_size(B, Sq, Sk, Hq, Hkv, d, int(num_splits)))
        workspace = _workspace(workspace, q, need)
        code = lib.fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B,
                                  Sq, Sk, Hq, Hkv, d, int(bool(causal)), float(scale), _dtype_code(q),
                                  int(num_splits), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _raise(code, "fa_fwd_splitkv")
    return out, lse


def fa_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                  seqused_k=None, causal: bool = False, scale: float | None = None, out=None, lse=None,
                  stream=None):
    """Forward over packed variable-length sequences.  q [total_q,Hq,d], k/v
    [total_k,Hkv,d], cu_seqlens_* int32 CUDA [B+1], seqused_k int32 CUDA [B] or None
    -> (o [total_q,Hq,d], lse [Hq,total_q] fp32)."""
    _check(q, "q")
    _check(k, "k", q.dtype)
    _check(v, "v", q.dtype)
    _check_kv(q, k, v, packed=True)
    total_q, Hq, d = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    B = _check_seqlens(q, cu_seqlens_q, cu_seqlens_k, seqused_k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(Hq, total_q, dtype=torch.float32, device=q.device)
    _check(out, "out", q.dtype)
    _check(lse, "lse", torch.float32)
    _shape(out, "out", q.shape)
    _shape(lse, "lse", (Hq, total_q))
    _same_device(q, k=k, v=v, out=out, lse=lse)
    with torch.cuda.device(q.device):
        code = _lib.load().fa_fwd_varlen(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), cu_seqlens_q.data_ptr(),
            cu_seqlens_k.data_ptr(), seqused_k.data_ptr() if seqused_k is not None else None, B,
            int(max_seqlen_q), int(max_seqlen_k), total_q, total_k, Hq, Hkv, d, int(bool(causal)),
            float(scale), _dtype_code(q), _stream_ptr(stream))
    _raise(code, "fa_fwd_varlen")
    return out, lse


def _check_seqlens(q, cu_seqlens_q, cu_seqlens_k, seqused_k) -> int:
    """Validates the sequence-boundary arrays of a packed batch; returns B."""
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)) + (
            (("seqused_k", seqused_k),) if seqused_k is not None else ()):
        if not isinstance(t, torch.Tensor) or t.device != q.device or t.dtype != torch.int32 or \
                not t.is_contiguous():
            raise ValueError(f"fa: {name} must be a contiguous int32 tensor on {q.device}")
    B = cu_seqlens_q.numel() - 1
    if B < 1 or cu_seqlens_k.numel() != B + 1 or (seqused_k is not None and seqused_k.numel() != B):
        raise ValueError("fa: cu_seqlens_q / cu_seqlens_k need B+1 entries, seqused_k B")
    return B


def _check_bwd_tensors(q, k, v, o, lse, dout, dq, dk, dv, lse_shape):
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq), ("dk", dk),
                    ("dv", dv)):
        _check(t, name, q.dtype)
    _check(lse, "lse", torch.float32)
    for name, t in (("o", o), ("dout", dout), ("dq", dq)):
        _shape(t, name, q.shape)
    _shape(dk, "dk", k.shape)
    _shape(dv, "dv", k.shape)
    _shape(lse, "lse", lse_shape)
    _same_device(q, k=k, v=v, o=o, lse=lse, dout=dout, dq=dq, dk=dk, dv=dv)


def fa_bwd_workspace_size(B: int, Sq: int, Hq: int, d: int) -> int:
    return int(_lib.load().fa_bwd_workspace_size(B, Sq, Hq, d))


def fa_bwd(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None,
           dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward. Returns (dq, dk, dv) in the input dtype."""
    _check(q, "q")
    _check_kv(q, k, v, packed=False)
    B, Sq, Hq, d = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check_bwd_tensors(q, k, v, o, lse, dout, dq, dk, dv, (B, Hq, Sq))
    with torch.cuda.device(q.device):
        workspace = _workspace(workspace, q, fa_bwd_workspace_size(B, Sq, Hq, d))
        code = _lib.load().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                  lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                  dv.data_ptr(), B, Sq, Sk, Hq, Hkv, d, int(bool(causal)),
                                  float(scale), _dtype_code(q), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _raise(code, "fa_bwd")
    return dq, dk, dv


def fa_bwd_varlen(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                  max_seqlen_k: int, seqused_k=None, causal: bool = False, scale: float | None = None,
                  dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward over packed variable-length sequences (layouts as fa_fwd_varlen)
    -> (dq [total_q,Hq,d], dk, dv [total_k,Hkv,d])."""
    _check(q, "q")
    _check_kv(q, k, v, packed=True)
    total_q, Hq, d = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    B = _check_seqlens(q, cu_seqlens_q, cu_seqlens_k, seqused_k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check_bwd_tensors(q, k, v, o, lse, dout, dq, dk, dv, (Hq, total_q))
    with torch.cuda.device(q.device):
        workspace = _workspace(workspace, q, fa_bwd_workspace_size(B, int(max_seqlen_q), Hq, d))
        code = _lib.load().fa_bwd_varlen(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
            seqused_k.data_ptr() if seqused_k is not None else None, B, int(max_seqlen_q), int(max_seqlen_k),
            total_q, total_k, Hq, Hkv, d, int(bool(causal)), float(scale), _dtype_code(q), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _raise(code, "fa_bwd_varlen")
    return dq, dk, dv


def fa_bwd_noalloc(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None,
                   dq=None, dk=None, dv=None, stream=None):
    """Backward without a workspace: the library keeps the scratch in a fixed device
    array (for callers that cannot allocate device memory).  Calls that overlap on
    the GPU race on that array.  Output tensors may be passed in to avoid allocating
    them here too.  Returns (dq, dk, dv)."""
    _check(q, "q")
    _check_kv(q, k, v, packed=False)
    B, Sq, Hq, d = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check_bwd_tensors(q, k, v, o, lse, dout, dq, dk, dv, (B, Hq, Sq))
    with torch.cuda.device(q.device):
        code = _lib.load().fa_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                          lse.data_ptr(), dout.data_ptr(), dq.data_ptr(),
                                          dk.data_ptr(), dv.data_ptr(), B, Sq, Sk, Hq, Hkv, d,
                                          int(bool(causal)), float(scale), _dtype_code(q),
                                          _stream_ptr(stream))
    _raise(code, "fa_bwd_noalloc")
    return dq, dk, dv


def fa_kv_cache_size(num_pages: int, page_size: int, Hkv: int, d: int, fmt: int = FA_KV_16) -> int:
    """Bytes of one pool of the paged cache (keys or values); 0 for unsupported sizes."""
    return int(_lib.load().fa_kv_cache_size(num_pages, page_size, Hkv, d, fmt))


class _Here:
    """Stands for torch.cuda.device(...) where that device is current already: the paged
    calls are a few microseconds on the GPU, and switching costs as much on the host."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _on(device, stream=None):
    """Makes `device` current, and `stream` if one is given: what a call allocates then
    belongs to the stream that it runs on, so its memory is not handed out again while
    that stream still uses it."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            handle = _stream_ptr(stream)  # 0 and 1 both name the legacy default stream
            stream = torch.cuda.ExternalStream(handle, device=device) if handle > 1 else \
                torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"fa: the stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    return _HERE if torch._C._cuda_getDevice() == device.index else torch.cuda.device(device)


def _check_index(t, name, shape, device):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"fa: {name} must be a contiguous int32 tensor on {device}")
    if t.shape != shape:
        raise ValueError(f"fa: {name} has shape {tuple(t.shape)}, expected {shape}")


def _check_cache(k_cache, v_cache, dtype, block_table, device):
    """Validates a pair of pools and their block table; returns (num_pages, Hkv,
    page_size, d, fmt, B, max_pages).  Pools are [num_pages, Hkv, page_size, d] in the
    call's dtype, or uint8 [num_pages, Hkv, page_size, 5 d / 8]."""
    for t in (k_cache, v_cache):
        if not isinstance(t, torch.Tensor) or t.device != device or not t.is_contiguous():
            raise ValueError(f"fa: k_cache and v_cache must be contiguous tensors on {device}")
    shape, kind = k_cache.shape, k_cache.dtype
    if v_cache.dtype != kind or (kind != dtype and kind != torch.uint8):
        raise ValueError(f"fa: the pools have dtypes {kind} and {v_cache.dtype}, expected {dtype} or uint8")
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("fa: k_cache and v_cache must be [num_pages, Hkv, page_size, d] (4-bit: 5 d / 8 bytes)")
    num_pages, Hkv, page_size, width = shape
    fmt = FA_KV_16
    if kind == torch.uint8:
        if width % 5:
            raise ValueError(f"fa: a 4-bit pool has 5 d / 8 bytes per token, got {width}")
        width, fmt = width * 8 // 5, FA_KV_INT4
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2 or block_table.dtype != torch.int32 or \
            block_table.device != device or not block_table.is_contiguous():
        raise ValueError(f"fa: block_table must be a contiguous int32 [B, max_pages] tensor on {device}")
    B, max_pages = block_table.shape
    return num_pages, Hkv, page_size, width, fmt, B, max_pages


def _token_rows(t, name, total, H, d, dtype, device):
    """A packed [total, H, d] tensor whose rows may lie apart (a slice of a fused
    projection); returns the distance between rows in elements."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"fa: {name} must be a tensor on {device}")
    if t.shape != (total, H, d) or t.dtype != dtype:
        raise ValueError(f"fa: {name} is {tuple(t.shape)} of {t.dtype}, expected {(total, H, d)} of {dtype}")
    row, head, one = t.stride()
    if one != 1 or (H > 1 and head != d):
        raise ValueError(f"fa: the heads of a row of {name} must be contiguous")
    return row if total > 1 else H * d


def fa_kv_append(q, k, v, k_cache, v_cache, cu_seqlens, seqlens_k, block_table, inv_freq=None,
                 interleaved: bool = False, q_out=None, stream=None):
    """Appends a step's packed tokens to a paged cache: rotates q [total,Hq,d] and k
    [total,Hkv,d] by their positions (pairs of the first 2 * len(inv_freq) head dims;
    inv_freq float32 CUDA or None) and writes k and v to their pages.  cu_seqlens [B+1]:
    the new tokens per sequence; seqlens_k [B]: its cached tokens, the new ones included;
    block_table [B,max_pages].  q, k, v may be slices of a fused projection.  q may be
    None.  Returns the rotated q [total,Hq,d]."""
    if not isinstance(k, torch.Tensor) or not k.is_cuda or k.dim() != 3:
        raise ValueError("fa: k must be a CUDA tensor [total, Hkv, d]")
    device, dtype, total = k.device, k.dtype, k.shape[0]
    dt = _dtype_code(k)
    num_pages, Hkv, page_size, d, fmt, B, max_pages = _check_cache(k_cache, v_cache, dtype, block_table, device)
    _check_index(cu_seqlens, "cu_seqlens", (B + 1,), device)
    _check_index(seqlens_k, "seqlens_k", (B,), device)
    k_stride = _token_rows(k, "k", total, Hkv, d, dtype, device)
    v_stride = _token_rows(v, "v", total, Hkv, d, dtype, device)
    Hq, q_stride = Hkv, Hkv * d
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("fa: q must be [total, Hq, d]")
        Hq = q.shape[1]
        q_stride = _token_rows(q, "q", total, Hq, d, dtype, device)
        if q_out is not None:
            _check(q_out, "q_out", dtype)
            _shape(q_out, "q_out", (total, Hq, d))
            _same_device(k, q_out=q_out)
    elif q_out is not None:
        raise ValueError("fa: q_out without q")
    rot = 0
    if inv_freq is not None:
        _check(inv_freq, "inv_freq", torch.float32)
        rot = 2 * inv_freq.numel()
        _same_device(k, inv_freq=inv_freq)
    with _on(device, stream):
        if q is not None and q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        code = _lib.load().fa_kv_append(
            q.data_ptr() if q is not None else None, k.data_ptr(), v.data_ptr(), q_stride, k_stride, v_stride,
            q_out.data_ptr() if q is not None else None, k_cache.data_ptr(), v_cache.data_ptr(),
            cu_seqlens.data_ptr(), seqlens_k.data_ptr(), block_table.data_ptr(),
            inv_freq.data_ptr() if rot else None, rot, 1 if interleaved else 0, B, total, Hq, Hkv, d, page_size,
            num_pages, max_pages, fmt, dt, _stream_ptr(stream))
    _raise(code, "fa_kv_append")
    return q_out


def fa_kv_gather(k_cache, v_cache, cu_seqlens_k, block_table, total_k: int, dtype=None, k=None, v=None,
                 stream=None):
    """Reads the first cu_seqlens_k[b+1] - cu_seqlens_k[b] cached tokens of every sequence
    back as packed rows -> (k, v) [total_k,Hkv,d].  dtype: the type of a 4-bit pool's
    scales and of its rows (a 16-bit pool has its own)."""
    _check(k_cache, "k_cache")
    if k_cache.dtype != torch.uint8:
        dtype = k_cache.dtype if dtype is None else dtype
    elif dtype is None:
        raise ValueError("fa: a 4-bit pool needs the dtype of its scales")
    device = k_cache.device
    num_pages, Hkv, page_size, d, fmt, B, max_pages = _check_cache(k_cache, v_cache, dtype, block_table, device)
    _check_index(cu_seqlens_k, "cu_seqlens_k", (B + 1,), device)
    total_k = int(total_k)
    shape = (total_k, Hkv, d)
    dt = _dtype_code(dtype)
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            _check(t, name, dtype)
            _shape(t, name, shape)
            _same_device(k_cache, **{name: t})
    with _on(device, stream):
        k = k_cache.new_empty(shape, dtype=dtype) if k is None else k
        v = k_cache.new_empty(shape, dtype=dtype) if v is None else v
        code = _lib.load().fa_kv_gather(k_cache.data_ptr(), v_cache.data_ptr(), k.data_ptr(), v.data_ptr(),
                                        cu_seqlens_k.data_ptr(), block_table.data_ptr(), B, total_k, Hkv, d,
                                        page_size, num_pages, max_pages, fmt, dt, _stream_ptr(stream))
    _raise(code, "fa_kv_gather")
    return k, v


def fa_fwd_paged_workspace_size(B: int, max_seqlen_q: int, Hq: int, Hkv: int, d: int) -> int:
    return int(_lib.load().fa_fwd_paged_workspace_size(B, max_seqlen_q, Hq, Hkv, d))


@functools.lru_cache(maxsize=256)
def _paged_workspace_size(device_index, B, max_seqlen_q, Hq, Hkv, d) -> int:
    """fa_fwd_paged_workspace_size on the current device, `device_index`."""
    return max(256, fa_fwd_paged_workspace_size(B, max_seqlen_q, Hq, Hkv, d))


def fa_fwd_paged(q, k_cache, v_cache, cu_seqlens_q, seqlens_k, block_table, max_seqlen_q: int,
                 causal: bool = False, scale: float | None = None, out=None, lse=None, workspace=None,
                 stream=None):
    """Forward over a paged cache (decoding and short chunks).  q [total_q,Hq,d], pools
    as fa_kv_append fills them, seqlens_k [B] cached tokens per sequence
    -> (o [total_q,Hq,d], lse [Hq,total_q] fp32)."""
    _check(q, "q")
    if q.dim() != 3:
        raise ValueError("fa: q must be [total_q, Hq, d]")
    total_q, Hq, d = q.shape
    device, dtype, max_seqlen_q = q.device, q.dtype, int(max_seqlen_q)
    dt = _dtype_code(q)
    num_pages, Hkv, page_size, dk, fmt, B, max_pages = _check_cache(k_cache, v_cache, dtype, block_table, device)
    _check_index(cu_seqlens_q, "cu_seqlens_q", (B + 1,), device)
    _check_index(seqlens_k, "seqlens_k", (B,), device)
    if dk != d:
        raise ValueError(f"fa: the pools hold head_dim {dk}, q has {d}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is not None:
        _check(out, "out", dtype)
        _shape(out, "out", q.shape)
    if lse is not None:
        _check(lse, "lse", torch.float32)
        _shape(lse, "lse", (Hq, total_q))
    if out is not None or lse is not None:
        _same_device(q, out=out, lse=lse)
    lib = _lib.load()
    with _on(device, stream):
        if out is None:
            out = torch.empty_like(q)
        if lse is None:
            lse = q.new_empty((Hq, total_q), dtype=torch.float32)
        need = _paged_workspace_size(device.index, B, max_seqlen_q, Hq, Hkv, d)
        if workspace is None:
            workspace = q.new_empty(need, dtype=torch.uint8)
        else:
            workspace = _workspace(workspace, q, need)
        code = lib.fa_fwd_paged(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
                                lse.data_ptr(), cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(),
                                block_table.data_ptr(), B, max_seqlen_q, total_q, Hq, Hkv, d, page_size,
                                num_pages, max_pages, fmt, 1 if causal else 0, float(scale), dt,
                                workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                _stream_ptr(stream))
    _raise(code, "fa_fwd_paged")
    return out, lse


def fa_last_device_status(stream=None):
    """(code, detail) of the device status word; synchronises the stream."""
    detail = ctypes.c_uint32(0)
    code = _lib.load().fa_last_device_status(_stream_ptr(stream), ctypes.byref(detail))
    return int(code), int(detail.value)


def fa_clear_device_status(stream=None):
    _raise(_lib.load().fa_clear_device_status(_stream_ptr(stream)), "fa_clear_device_status")


def fa_set_unit_schedule(mode: int):
    """Forward unit order: FA_SCHED_STATIC (persistent grid, fixed stride),
    FA_SCHED_CLC (one CTA per unit, running CTAs cancel pending ones to take their
    units) or FA_SCHED_AUTO (the default: CLC for causal launches over >= 4096 keys,
    else STATIC).  Process-wide."""
    _raise(_lib.load().fa_set_unit_schedule(int(mode)), "fa_set_unit_schedule")


def fa_set_exp2_emulation(pairs_of_4: int):
    """Forward exp2 split: how many of every four pairs of exponentials of an unmasked
    score tile use the FMA-pipe cubic instead of the special-function unit (0..3), or
    -1 for the library's per-head-dim default.  Process-wide."""
    _raise(_lib.load().fa_set_exp2_emulation(int(pairs_of_4)), "fa_set_exp2_emulation")


def fa_set_wait_timeout_ms(ms: int):
    """Limit (ms, 1..600000; 1000 initially) after which a kernel's pipeline wait gives
    up and reports FA_ERR_DEVICE_TIMEOUT.  Wall-clock time on the device: raise it on
    GPUs time-sliced between processes.  Process-wide."""
    _raise(_lib.load().fa_set_wait_timeout_ms(int(ms)), "fa_set_wait_timeout_ms")


def fa_debug_inject(mode: int):
    _raise(_lib.load().fa_debug_inject(int(mode)), "fa_debug_inject")


def fa_debug_exp2(x, mode: int = 0, stream=None):
    """The kernels' exp2 on a CUDA fp32 tensor: mode 0 the FMA-pipe cubic, 1 the SFU
    instruction.  Returns a new tensor (enqueued on the stream)."""
    if x.device.type != "cuda" or x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA float32 tensor")
    y = torch.empty_like(x)
    _raise(_lib.load().fa_debug_exp2(x.data_ptr(), y.data_ptr(), x.numel(), int(mode), _stream_ptr(stream)),
           "fa_debug_exp2")
    return y
