"""ctypes binding of libfa.so (include/fa.h), argument marshalling only.

Every step of the attention path runs in the CUDA kernels behind the C ABI;
this module checks tensor properties, allocates outputs and workspace with
PyTorch when the caller does not pass them, and forwards raw device pointers
and the current CUDA stream. There is no fallback: if the library is missing
or a call fails, an exception is raised.

``stream`` names another stream (of the current device) to run on. Outputs and
workspaces that the call allocates are then that stream's for the allocator, as
inside ``with torch.cuda.stream(stream)``: their memory is not handed on while
kernels on it still run.
"""

from __future__ import annotations

import ctypes
import math
import os
import re
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "fa.h")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_NO_BLOCKS = range(6)
FA_BF16, FA_FP32 = 0, 1


class FAError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} ({code})")


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfa.so and declare the C signatures. Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    vp, sz, i, f = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    lib.fa_fwd_workspace_size.argtypes = [i, i, i, i]
    lib.fa_fwd_workspace_size.restype = sz
    lib.fa_bwd_workspace_size.argtypes = [i, i, i, i]
    lib.fa_bwd_workspace_size.restype = sz
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp, i, vp, sz, vp]
    lib.fa_fwd.restype = i
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp, i, vp, sz, vp]
    lib.fa_bwd.restype = i
    lib.fa_fwd_varlen_workspace_size.argtypes = [i, i, i]
    lib.fa_fwd_varlen_workspace_size.restype = sz
    lib.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, sz, vp]
    lib.fa_fwd_varlen.restype = i
    lib.fa_bwd_varlen_workspace_size.argtypes = [i, i, i, i]
    lib.fa_bwd_varlen_workspace_size.restype = sz
    lib.fa_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, sz, vp]
    lib.fa_bwd_varlen.restype = i
    lib.fa_decode_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.fa_decode_workspace_size.restype = sz
    lib.fa_decode.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, i, i, vp, sz, vp]
    lib.fa_decode.restype = i
    lib.fa_fwd_fp8_workspace_size.argtypes = [i, i, i, i]
    lib.fa_fwd_fp8_workspace_size.restype = sz
    lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp, vp, sz, vp]
    lib.fa_fwd_fp8.restype = i
    lib.fa_cache_plan.argtypes = [vp] * 9 + [i] * 5 + [vp, sz, vp]
    lib.fa_cache_plan.restype = i
    lib.fa_cache_append.argtypes = [vp] * 7 + [i] * 5 + [vp]
    lib.fa_cache_append.restype = i
    lib.fa_fwd_paged_workspace_size.argtypes = [i] * 6
    lib.fa_fwd_paged_workspace_size.restype = sz
    lib.fa_fwd_paged.argtypes = [vp] * 10 + [i] * 9 + [f, i, vp, sz, vp]
    lib.fa_fwd_paged.restype = i
    lib.fa_fwd_paged_prefix_workspace_size.argtypes = [i] * 7
    lib.fa_fwd_paged_prefix_workspace_size.restype = sz
    lib.fa_fwd_paged_prefix.argtypes = [vp] * 13 + [i] * 11 + [f, i, vp, sz, vp]
    lib.fa_fwd_paged_prefix.restype = i
    lib.fa_qk_norm_rope.argtypes = [vp] * 6 + [f, vp, i, i, vp, vp] + [i] * 6 + [vp]
    lib.fa_qk_norm_rope.restype = i
    lib.fa_qk_norm_rope_bwd_workspace_size.argtypes = [i]
    lib.fa_qk_norm_rope_bwd_workspace_size.restype = sz
    lib.fa_qk_norm_rope_bwd.argtypes = [vp] * 10 + [f, vp, i, i, vp, vp] + [i] * 6 + [vp, sz, vp]
    lib.fa_qk_norm_rope_bwd.restype = i
    lib.fa_qk_norm_rope_append.argtypes = [vp] * 11 + [f, vp, i, i, vp, vp] + [i] * 7 + [vp]
    lib.fa_qk_norm_rope_append.restype = i
    u64 = ctypes.c_ulonglong
    lib.fa_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, f, u64, vp, sz, vp]
    lib.fa_fwd_dropout.restype = i
    lib.fa_bwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, f, u64, vp, sz, vp]
    lib.fa_bwd_dropout.restype = i
    lib.fa_get_status.argtypes = [vp, vp]
    lib.fa_get_status.restype = i
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_last_launch_count.argtypes = []
    lib.fa_last_launch_count.restype = i
    lib.fa_set_timing_events.argtypes = [vp, vp]
    lib.fa_set_timing_events.restype = i
    lib.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp, i, vp]
    lib.fa_bwd_noalloc.restype = i
    lib.fa_bwd_noalloc_get_status.argtypes = [vp]
    lib.fa_bwd_noalloc_get_status.restype = i
    _lib = lib
    return lib


def declared_functions(header: str = HEADER_PATH):
    """Names of the functions include/fa.h declares."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(fa_[a-z0-9_]+)\s*\(", text)))


def status_string(code: int) -> str:
    return load().fa_status_string(code).decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# the current stream's handle without a Stream object (a microsecond or two of
# a decoding call's host time)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# the current device of a process that has CUDA tensors
_device_index = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_handle(stream: Optional[torch.cuda.Stream]):
    if stream is not None:
        if stream.device_index != torch.cuda.current_device():
            raise ValueError(f"the stream is on {stream.device} but the current device is"
                             f" cuda:{torch.cuda.current_device()}")
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_device_index())


def _check_device(q: torch.Tensor):
    """The kernels run on the current CUDA device: q must live there."""
    if not q.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if q.get_device() != _device_index():
        raise ValueError(f"tensors are on {q.device} but the current device is cuda:{torch.cuda.current_device()}:"
                         " call under torch.cuda.device(q.device)")


def _in(t: torch.Tensor, shape, dtype, device, name: str) -> torch.Tensor:
    """Check a buffer the kernels read or write as exactly `shape` contiguous
    elements of `dtype` on `device` (the library cannot see its size)."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t
    raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on {device}")


def _out(t: Optional[torch.Tensor], shape, dtype, device, name: str, stream=None) -> torch.Tensor:
    """A caller-supplied output, checked as in _in, or a new one of `stream`."""
    if t is None:
        if stream is None:
            return torch.empty(tuple(shape), dtype=dtype, device=device)
        with torch.cuda.stream(stream):
            return torch.empty(tuple(shape), dtype=dtype, device=device)
    return _in(t, shape, dtype, device, name)


def _ws(ws: Optional[torch.Tensor], nbytes, device, stream=None) -> torch.Tensor:
    """A caller-supplied workspace (on the device, contiguous; its size is
    checked by the library) or a new one of `nbytes`, of `stream`."""
    if ws is None:
        nbytes = nbytes() if callable(nbytes) else nbytes
        if stream is None:
            return workspace(nbytes, device)
        with torch.cuda.stream(stream):
            return workspace(nbytes, device)
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous tensor on {device}")
    return ws


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _check_qkv(*ts: torch.Tensor):
    q = ts[0]
    _check_device(q)
    for t in ts:
        if t.device != q.device:
            raise ValueError("tensors must be on the same CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous [B, H, N, d]")
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError("q, k, v (and o, dO) must share shape and dtype")
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    if q.dtype == torch.bfloat16:
        return FA_BF16
    if q.dtype == torch.float32:
        return FA_FP32
    raise ValueError("dtype must be bfloat16 or float32")


def _mask_ptrs(blockmask, kv_len, q):
    if blockmask is not None:
        T = q.shape[2] // 128
        if blockmask.dtype != torch.uint8 or blockmask.shape != (T, T) or not blockmask.is_contiguous():
            raise ValueError(f"blockmask must be a contiguous uint8 [{T}, {T}] tensor")
        if blockmask.device != q.device:
            raise ValueError("blockmask must be on the same device")
    if kv_len is not None:
        if kv_len.dtype != torch.int32 or kv_len.shape != (q.shape[0],) or kv_len.device != q.device:
            raise ValueError("kv_len must be an int32 [B] tensor on the same device")
    return _ptr(blockmask), _ptr(kv_len)


def fwd_workspace_size(B, H, N, d) -> int:
    return load().fa_fwd_workspace_size(B, H, N, d)


def bwd_workspace_size(B, H, N, d) -> int:
    return load().fa_bwd_workspace_size(B, H, N, d)


def fwd_varlen_workspace_size(H, total, d) -> int:
    return load().fa_fwd_varlen_workspace_size(H, total, d)


def bwd_varlen_workspace_size(B, H, total, d) -> int:
    return load().fa_bwd_varlen_workspace_size(B, H, total, d)


def decode_workspace_size(B, H, Nq, Nk, d, num_splits: int = 0) -> int:
    return load().fa_decode_workspace_size(B, H, Nq, Nk, d, num_splits)


def fwd_fp8_workspace_size(B, H, N, d) -> int:
    return load().fa_fwd_fp8_workspace_size(B, H, N, d)


def fwd_paged_workspace_size(B, Hq, Hkv, total, max_new, d) -> int:
    return load().fa_fwd_paged_workspace_size(B, Hq, Hkv, total, max_new, d)


def workspace(nbytes: int, device) -> torch.Tensor:
    """A device buffer usable as workspace (256-byte aligned by the allocator)."""
    return torch.empty(max(256, nbytes), dtype=torch.uint8, device=device)


def forward(q, k, v, scale: Optional[float] = None, causal: bool = False, blockmask=None, kv_len=None,
            out=None, lse=None, ws=None, stream=None):
    """O, L = fa_fwd(...). Returns (o [B,H,N,d], lse fp32 [B,H,N])."""
    lib = load()
    dtype = _check_qkv(q, k, v)
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = _out(out, q.shape, q.dtype, q.device, "out", stream)
    L = _out(lse, (B, H, N), torch.float32, q.device, "lse", stream)
    ws = _ws(ws, lambda: lib.fa_fwd_workspace_size(B, H, N, d) if dtype == FA_FP32 else 256, q.device, stream)
    bm, kl = _mask_ptrs(blockmask, kv_len, q)
    rc = lib.fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(L), B, H, N, d, scale, int(bool(causal)), bm, kl,
                    dtype, _ptr(ws), _nbytes(ws), _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd")
    return o, L


def _check_packed(cu_seqlens, *ts: torch.Tensor):
    q = ts[0]
    _check_device(q)
    for t in ts:
        if t.device != q.device:
            raise ValueError("tensors must be on the same CUDA device")
        if not t.is_contiguous() or t.dim() != 3:
            raise ValueError("packed tensors must be contiguous [total, H, d]")
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError("packed q, k, v (and o, dO) must share shape and dtype")
    if q.dtype != torch.bfloat16:
        raise ValueError("packed variable-length batches are bfloat16 only")
    if (cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2
            or cu_seqlens.device != q.device or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens must be a contiguous int32 [B + 1] tensor on the same device")
    return FA_BF16


def forward_varlen(q, k, v, cu_seqlens, max_seqlen: int, scale: Optional[float] = None, causal: bool = False,
                   out=None, lse=None, ws=None, stream=None):
    """O, L = fa_fwd_varlen(...) on a packed batch. q, k, v: [total, H, d]
    bf16; cu_seqlens: int32 [B + 1] offsets on the device; max_seqlen: the
    longest sequence. Returns (o [total, H, d], lse fp32 [H, total])."""
    lib = load()
    dtype = _check_packed(cu_seqlens, q, k, v)
    total, H, d = q.shape
    B = cu_seqlens.numel() - 1
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = _out(out, q.shape, q.dtype, q.device, "out", stream)
    L = _out(lse, (H, total), torch.float32, q.device, "lse", stream)
    ws = _ws(ws, lambda: lib.fa_fwd_varlen_workspace_size(H, total, d), q.device, stream)
    rc = lib.fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(L), _ptr(cu_seqlens), B, H, total,
                           int(max_seqlen), d, scale, int(bool(causal)), dtype, _ptr(ws), _nbytes(ws),
                           _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_varlen")
    return o, L


def backward_varlen(q, k, v, o, lse, do, cu_seqlens, max_seqlen: int, scale: Optional[float] = None,
                    causal: bool = False, dq=None, dk=None, dv=None, ws=None, stream=None):
    """dQ, dK, dV = fa_bwd_varlen(...) on a packed batch ([total, H, d] bf16;
    lse fp32 [H, total] from forward_varlen). Returns (dq, dk, dv)."""
    lib = load()
    dtype = _check_packed(cu_seqlens, q, k, v, o, do)
    total, H, d = q.shape
    B = cu_seqlens.numel() - 1
    _in(lse, (H, total), torch.float32, q.device, "lse")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = _out(dq, q.shape, q.dtype, q.device, "dq", stream)
    dk = _out(dk, q.shape, q.dtype, q.device, "dk", stream)
    dv = _out(dv, q.shape, q.dtype, q.device, "dv", stream)
    ws = _ws(ws, lambda: lib.fa_bwd_varlen_workspace_size(B, H, total, d), q.device, stream)
    rc = lib.fa_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                           _ptr(cu_seqlens), B, H, total, int(max_seqlen), d, scale, int(bool(causal)), dtype,
                           _ptr(ws), _nbytes(ws), _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_bwd_varlen")
    return dq, dk, dv


def forward_fp8(q, k, v, signs, scale: Optional[float] = None, causal: bool = False, kv_len=None, out=None,
                lse=None, ws=None, stream=None):
    """O, L = fa_fwd_fp8(...): the FP8 forward pass with a Hadamard rotation
    (signs: float32 [128] of +-1 on the device; None skips the rotation) and
    per-block scales. q, k, v: [B, H, N, 128] bf16. Returns (o bf16, lse fp32
    [B, H, N])."""
    lib = load()
    dtype = _check_qkv(q, k, v)
    if dtype != FA_BF16:
        raise ValueError("the FP8 path takes bfloat16 inputs")
    B, H, N, d = q.shape
    if signs is not None and (signs.dtype != torch.float32 or signs.shape != (d,) or signs.device != q.device):
        raise ValueError("signs must be None or a float32 [d] tensor on the same device")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = _out(out, q.shape, q.dtype, q.device, "out", stream)
    L = _out(lse, (B, H, N), torch.float32, q.device, "lse", stream)
    ws = _ws(ws, lambda: lib.fa_fwd_fp8_workspace_size(B, H, N, d), q.device, stream)
    _, kl = _mask_ptrs(None, kv_len, q)
    rc = lib.fa_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(L), B, H, N, d, scale, int(bool(causal)), kl,
                        _ptr(signs), _ptr(ws), _nbytes(ws), _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_fp8")
    return o, L


def forward_dropout(q, k, v, dropout_p: float, seed: int, scale: Optional[float] = None, causal: bool = False,
                    kv_len=None, out=None, lse=None, ws=None, stream=None):
    """O, L = fa_fwd_dropout(...): attention with dropout on the
    probabilities (bf16 [B, H, N, d]). Returns (o, lse)."""
    lib = load()
    if _check_qkv(q, k, v) != FA_BF16:
        raise ValueError("dropout takes bfloat16 inputs")
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = _out(out, q.shape, q.dtype, q.device, "out", stream)
    L = _out(lse, (B, H, N), torch.float32, q.device, "lse", stream)
    ws = _ws(ws, 256, q.device, stream)
    _, kl = _mask_ptrs(None, kv_len, q)
    rc = lib.fa_fwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(L), B, H, N, d, scale, int(bool(causal)), kl,
                            float(dropout_p), int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(ws), _nbytes(ws),
                            _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_dropout")
    return o, L


def backward_dropout(q, k, v, o, lse, do, dropout_p: float, seed: int, scale: Optional[float] = None,
                     causal: bool = False, kv_len=None, dq=None, dk=None, dv=None, ws=None, stream=None):
    """dQ, dK, dV = fa_bwd_dropout(...) for forward_dropout's outputs."""
    lib = load()
    if _check_qkv(q, k, v, o, do) != FA_BF16:
        raise ValueError("dropout takes bfloat16 inputs")
    B, H, N, d = q.shape
    _in(lse, (B, H, N), torch.float32, q.device, "lse")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = _out(dq, q.shape, q.dtype, q.device, "dq", stream)
    dk = _out(dk, q.shape, q.dtype, q.device, "dk", stream)
    dv = _out(dv, q.shape, q.dtype, q.device, "dv", stream)
    ws = _ws(ws, lambda: lib.fa_bwd_workspace_size(B, H, N, d), q.device, stream)
    _, kl = _mask_ptrs(None, kv_len, q)
    rc = lib.fa_bwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                            B, H, N, d, scale, int(bool(causal)), kl, float(dropout_p),
                            int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(ws), _nbytes(ws), _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_bwd_dropout")
    return dq, dk, dv


def decode(q, k_cache, v_cache, cache_len=None, scale: Optional[float] = None, num_splits: int = 0, out=None,
           lse=None, ws=None, stream=None):
    """O, L = fa_decode(...): Nq (1..8) query rows per (b, h) against a
    [B, H, Nk, d] bf16 cache, keys split across CTAs and merged. Returns
    (o [B, H, Nq, d], lse fp32 [B, H, Nq])."""
    lib = load()
    _check_device(q)
    for t in (q, k_cache, v_cache):
        if t.device != q.device or not t.is_contiguous() or t.dim() != 4 or t.dtype != torch.bfloat16:
            raise ValueError("q and the cache must be contiguous bf16 [B, H, N, d] tensors on one CUDA device")
    B, H, Nq, d = q.shape
    if k_cache.shape != v_cache.shape or k_cache.shape[:2] != (B, H) or k_cache.shape[3] != d:
        raise ValueError("the cache must be [B, H, Nk, d] with q's B, H and d")
    Nk = k_cache.shape[2]
    if cache_len is not None and (cache_len.dtype != torch.int32 or cache_len.shape != (B,)
                                  or cache_len.device != q.device):
        raise ValueError("cache_len must be an int32 [B] tensor on the same device")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = _out(out, q.shape, q.dtype, q.device, "out", stream)
    L = _out(lse, (B, H, Nq), torch.float32, q.device, "lse", stream)
    ws = _ws(ws, lambda: lib.fa_decode_workspace_size(B, H, Nq, Nk, d, num_splits), q.device, stream)
    rc = lib.fa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(L), B, H, Nq, Nk, d, scale,
                       _ptr(cache_len), int(num_splits), FA_BF16, _ptr(ws), _nbytes(ws), _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_decode")
    return o, L


class _PagedCacheBuffers(NamedTuple):
    k: torch.Tensor            # float8_e4m3fn [num_blocks, Hkv, block_size, d]
    v: torch.Tensor
    k_scale: torch.Tensor      # float32 [num_blocks, Hkv]
    v_scale: torch.Tensor
    block_table: torch.Tensor  # int32 [B, max_blocks]
    cache_len: torch.Tensor    # int32 [B]
    free_blocks: torch.Tensor  # int32 [num_blocks], a ring
    free_state: torch.Tensor   # int32 [2]: its head and count


class PagedCache(_PagedCacheBuffers):
    """The buffers of a paged 8-bit cache and of the requests it serves, as
    cache_plan, cache_append and forward_paged take them; and, beside the
    tuple, `status` (uint8 [256]), cache_plan's workspace, read by get_status."""
    status: Optional[torch.Tensor] = None


def paged_cache(num_blocks: int, Hkv: int, block_size: int, d: int, B: int, max_blocks: int,
                device="cuda") -> PagedCache:
    """An empty cache of num_blocks blocks for up to B requests of at most
    max_blocks blocks each. The other layers of a model have k, v, k_scale and
    v_scale of their own and share the tables."""
    i32 = dict(dtype=torch.int32, device=device)
    k, v = (torch.zeros((num_blocks, Hkv, block_size, d), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
            for _ in range(2))
    ks, vs = (torch.zeros((num_blocks, Hkv), dtype=torch.float32, device=device) for _ in range(2))
    cache = PagedCache(k, v, ks, vs, torch.full((B, max_blocks), -1, **i32), torch.zeros(B, **i32),
                       torch.arange(num_blocks, **i32), torch.tensor([0, num_blocks], **i32))
    cache.status = torch.zeros(256, dtype=torch.uint8, device=device)
    return cache


def cache_plan(new_len, cache_len, block_table, free_blocks, free_state, block_size: int,
               total: Optional[int] = None, cache_len_out=None, free_state_out=None, cu_seqlens=None, slots=None,
               ws=None, stream=None):
    """cu_seqlens, slots = fa_cache_plan(...): blocks for each request's
    new_len tokens (-1 releases the request) and their slots. new_len,
    cache_len: int32 [B]; block_table: int32 [B, max_blocks]; free_blocks:
    int32 [num_blocks]; free_state: int32 [2]. cache_len and free_state are
    updated in place unless cache_len_out or free_state_out is given. total
    (the size of the packed batch) is needed when slots is not passed in.
    Whether every request got its blocks (FA_OK, FA_ERR_NO_BLOCKS or
    FA_ERR_INVALID_ARG) is read by get_status(ws), which waits for the stream:
    pass ws (a cache's `status`), as nothing reads a workspace of the call's
    own. On the device a refused request's tokens have slot -1; cu_seqlens
    lists them all the same, and forward_paged takes them for the last tokens
    that the cache holds.
    Returns (cu_seqlens int32 [B + 1], slots int32 [total])."""
    lib = load()
    _check_device(new_len)
    dev, i32 = new_len.device, torch.int32
    if new_len.dim() != 1 or block_table.dim() != 2 or free_blocks.dim() != 1:
        raise ValueError("expected new_len [B], block_table [B, max_blocks] and free_blocks [num_blocks]")
    B, max_blocks, num_blocks = new_len.numel(), block_table.shape[1], free_blocks.numel()
    _in(new_len, (B,), i32, dev, "new_len")
    _in(cache_len, (B,), i32, dev, "cache_len")
    _in(block_table, (B, max_blocks), i32, dev, "block_table")
    _in(free_blocks, (num_blocks,), i32, dev, "free_blocks")
    _in(free_state, (2,), i32, dev, "free_state")
    cache_len_out = cache_len if cache_len_out is None else _in(cache_len_out, (B,), i32, dev, "cache_len_out")
    free_state_out = free_state if free_state_out is None else _in(free_state_out, (2,), i32, dev, "free_state_out")
    if slots is None and total is None:
        raise ValueError("pass slots, or total, the size of the packed batch")
    total = slots.numel() if total is None else int(total)
    cu = _out(cu_seqlens, (B + 1,), i32, dev, "cu_seqlens", stream)
    slots = _out(slots, (total,), i32, dev, "slots", stream)
    ws = _ws(ws, 256, dev, stream)
    rc = lib.fa_cache_plan(_ptr(new_len), _ptr(cache_len), _ptr(cache_len_out), _ptr(block_table), _ptr(free_blocks),
                           _ptr(free_state), _ptr(free_state_out), _ptr(cu), _ptr(slots), B, max_blocks, num_blocks,
                           int(block_size), total, _ptr(ws), _nbytes(ws), _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_cache_plan")
    return cu, slots


def _check_paged(k_cache, v_cache, k_scale, v_scale, device):
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("the cache must be [num_blocks, Hkv, block_size, d]")
    e4m3, scales = torch.float8_e4m3fn, shape[:2]
    _in(k_cache, shape, e4m3, device, "k_cache")
    _in(v_cache, shape, e4m3, device, "v_cache")
    _in(k_scale, scales, torch.float32, device, "k_scale")
    _in(v_scale, scales, torch.float32, device, "v_scale")
    return shape


def cache_append(k, v, k_cache, v_cache, k_scale, v_scale, slots, stream=None):
    """fa_cache_append(...): quantises k, v [total, Hkv, d] bf16 into the rows
    `slots` (int32 [total], from cache_plan) of the caches (float8_e4m3fn
    [num_blocks, Hkv, block_size, d]; scales float32 [num_blocks, Hkv])."""
    lib = load()
    _check_device(k)
    num_blocks, H, bs, d = _check_paged(k_cache, v_cache, k_scale, v_scale, k.device)
    if k.dim() != 3:
        raise ValueError("k and v must be [total, Hkv, d]")
    total = k.shape[0]
    for t, name in ((k, "k"), (v, "v")):
        _in(t, (total, H, d), torch.bfloat16, k.device, name)
    _in(slots, (total,), torch.int32, k.device, "slots")
    rc = lib.fa_cache_append(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                             _ptr(slots), total, H, d, num_blocks, bs, _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_cache_append")


def forward_paged(q, k_cache, v_cache, k_scale, v_scale, cu_seqlens, cache_len, block_table, max_new: int,
                  scale: Optional[float] = None, causal: bool = True, out=None, lse=None, ws=None, stream=None):
    """O, L = fa_fwd_paged(...): attention of the packed new tokens q
    [total, Hq, d] bf16 over the paged cache, which holds them as well
    (cache_len counts them). max_new: the most new tokens of a request.
    Returns (o [total, Hq, d], lse fp32 [Hq, total])."""
    lib = load()
    _check_device(q)
    num_blocks, Hkv, bs, d = _check_paged(k_cache, v_cache, k_scale, v_scale, q.device)
    if q.dim() != 3 or block_table.dim() != 2 or cache_len.dim() != 1:
        raise ValueError("expected q [total, Hq, d], block_table [B, max_blocks] and cache_len [B]")
    total, Hq, _ = q.shape
    B, max_blocks = block_table.shape
    _in(q, (total, Hq, d), torch.bfloat16, q.device, "q")
    _in(cu_seqlens, (B + 1,), torch.int32, q.device, "cu_seqlens")
    _in(cache_len, (B,), torch.int32, q.device, "cache_len")
    _in(block_table, (B, max_blocks), torch.int32, q.device, "block_table")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = _out(out, q.shape, q.dtype, q.device, "out", stream)
    L = _out(lse, (Hq, total), torch.float32, q.device, "lse", stream)
    ws = _ws(ws, lambda: lib.fa_fwd_paged_workspace_size(B, Hq, Hkv, total, int(max_new), d), q.device, stream)
    rc = lib.fa_fwd_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(o), _ptr(L),
                          _ptr(cu_seqlens), _ptr(cache_len), _ptr(block_table), B, Hq, Hkv, total, int(max_new),
                          max_blocks, num_blocks, bs, d, scale, int(bool(causal)), _ptr(ws), _nbytes(ws),
                          _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_paged")
    return o, L


def backward(q, k, v, o, lse, do, scale: Optional[float] = None, causal: bool = False, blockmask=None,
             kv_len=None, dq=None, dk=None, dv=None, ws=None, stream=None):
    """dQ, dK, dV = fa_bwd(...). Returns (dq, dk, dv)."""
    lib = load()
    dtype = _check_qkv(q, k, v, o, do)
    B, H, N, d = q.shape
    _in(lse, (B, H, N), torch.float32, q.device, "lse")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = _out(dq, q.shape, q.dtype, q.device, "dq", stream)
    dk = _out(dk, q.shape, q.dtype, q.device, "dk", stream)
    dv = _out(dv, q.shape, q.dtype, q.device, "dv", stream)
    ws = _ws(ws, lambda: lib.fa_bwd_workspace_size(B, H, N, d), q.device, stream)
    bm, kl = _mask_ptrs(blockmask, kv_len, q)
    rc = lib.fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                    B, H, N, d, scale, int(bool(causal)), bm, kl, dtype, _ptr(ws), _nbytes(ws),
                    _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_bwd")
    return dq, dk, dv


def get_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronise and read (then clear) the device status word of a workspace."""
    return load().fa_get_status(_ptr(ws), _stream_handle(stream))


def last_launch_count() -> int:
    return load().fa_last_launch_count()


def set_timing_events(begin=None, end=None):
    """Record torch.cuda.Event `begin`/`end` around the main attention kernel
    of the following calls on this thread (None, None turns it off)."""
    b = None if begin is None else ctypes.c_void_p(begin.cuda_event)
    e = None if end is None else ctypes.c_void_p(end.cuda_event)
    rc = load().fa_set_timing_events(b, e)
    if rc != FA_OK:
        raise FAError(rc, "fa_set_timing_events")


def backward_noalloc(q, k, v, o, lse, do, scale: Optional[float] = None, causal: bool = False, blockmask=None,
                     kv_len=None, dq=None, dk=None, dv=None, stream=None):
    """dQ, dK, dV = fa_bwd_noalloc(...): the backward pass with the library's
    own fixed scratch instead of a workspace (for callers that cannot allocate
    device memory). Outputs are allocated here only if not passed in."""
    fn = load().fa_bwd_noalloc
    dtype = _check_qkv(q, k, v, o, do)
    B, H, N, d = q.shape
    _in(lse, (B, H, N), torch.float32, q.device, "lse")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = _out(dq, q.shape, q.dtype, q.device, "dq", stream)
    dk = _out(dk, q.shape, q.dtype, q.device, "dk", stream)
    dv = _out(dv, q.shape, q.dtype, q.device, "dv", stream)
    bm, kl = _mask_ptrs(blockmask, kv_len, q)
    rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d,
            scale, int(bool(causal)), bm, kl, dtype, _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_bwd_noalloc")
    return dq, dk, dv


def noalloc_status(stream=None) -> int:
    """Synchronise and read (then clear) the status word of the last
    fa_bwd_noalloc call on the current device (fa_bwd_noalloc_get_status)."""
    return load().fa_bwd_noalloc_get_status(_stream_handle(stream))


from . import paged_prefix as _prefix, qk_norm as _norm  # noqa: E402  (they use what stands above)

# The names of include/fa.h, bound to the wrappers above and in those modules
# (same arguments in tensor form; outputs returned rather than passed as pointers).
C_NAMES = {
    "fa_fwd": forward,
    "fa_bwd": backward,
    "fa_fwd_workspace_size": fwd_workspace_size,
    "fa_bwd_workspace_size": bwd_workspace_size,
    "fa_fwd_varlen": forward_varlen,
    "fa_bwd_varlen": backward_varlen,
    "fa_fwd_varlen_workspace_size": fwd_varlen_workspace_size,
    "fa_bwd_varlen_workspace_size": bwd_varlen_workspace_size,
    "fa_decode": decode,
    "fa_decode_workspace_size": decode_workspace_size,
    "fa_cache_plan": cache_plan,
    "fa_cache_append": cache_append,
    "fa_fwd_paged": forward_paged,
    "fa_fwd_paged_workspace_size": fwd_paged_workspace_size,
    "fa_fwd_paged_prefix": _prefix.forward_paged_prefix,
    "fa_fwd_paged_prefix_workspace_size": _prefix.fwd_paged_prefix_workspace_size,
    "fa_qk_norm_rope": _norm.qk_norm_rope,
    "fa_qk_norm_rope_bwd": _norm.qk_norm_rope_backward,
    "fa_qk_norm_rope_bwd_workspace_size": _norm.qk_norm_rope_bwd_workspace_size,
    "fa_qk_norm_rope_append": _norm.qk_norm_rope_append,
    "fa_fwd_fp8": forward_fp8,
    "fa_fwd_fp8_workspace_size": fwd_fp8_workspace_size,
    "fa_fwd_dropout": forward_dropout,
    "fa_bwd_dropout": backward_dropout,
    "fa_bwd_noalloc": backward_noalloc,
    "fa_bwd_noalloc_get_status": noalloc_status,
    "fa_get_status": get_status,
    "fa_status_string": status_string,
    "fa_last_launch_count": last_launch_count,
    "fa_set_timing_events": set_timing_events,
}
globals().update(C_NAMES)
