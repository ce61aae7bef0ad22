"""Binding of the per-head norm with rotation, its gradient and its form that
writes into the paged cache (fa_qk_norm_rope* of include/fa.h), as binding.py
binds the other calls."""

from __future__ import annotations

import struct

import torch

from . import binding as _b

_pack_rows = struct.Struct("@Pqqq").pack


def _rows(t: torch.Tensor) -> bytes:
    """A [B, H, N, d] or [total, H, d] view as an fa_rows, whose last dimension
    has been found contiguous."""
    s = t.stride()
    return _pack_rows(t.data_ptr(), s[0], s[1], s[2]) if len(s) == 4 else _pack_rows(t.data_ptr(), 0, s[1], s[0])


def _like(t, shape, dtype, device, name):
    """Check a tensor of rows of heads: any strides but the heads' own."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.stride(-1) == 1:
        return t
    raise ValueError(f"{name} must be a {dtype} {list(shape)} tensor on {device} with contiguous heads")


def _norm_sizes(q, k, inv_freq, q_weight, k_weight, cu_seqlens, ends):
    """Checks what the norm calls share (in few steps: a decoding call's host
    time is these); returns (B, N, Hq, Hkv, d, rot, type, shapes of q and k,
    dtype, device)."""
    _b._check_device(q)
    qs, ks, dtype, dev = q.shape, k.shape, q.dtype, q.device
    if cu_seqlens is not None:
        if len(qs) != 3 or len(ks) != 3:
            raise ValueError("expected packed q, k [total, H, d] with cu_seqlens")
        N, Hq, d = qs
        B, Hkv, same = cu_seqlens.numel() - 1, ks[1], ks[0] == N and ks[2] == d
        if B < 1:
            raise ValueError("cu_seqlens must be [B + 1]")
        _b._in(cu_seqlens, (B + 1,), torch.int32, dev, "cu_seqlens")
    else:
        if len(qs) != 4 or len(ks) != 4:
            raise ValueError("expected q, k [B, H, N, d], or [total, H, d] with cu_seqlens")
        B, Hq, N, d = qs
        Hkv, same = ks[1], ks[0] == B and ks[2] == N and ks[3] == d
    if dtype is torch.bfloat16:
        code = _b.FA_BF16
    elif dtype is torch.float32:
        code = _b.FA_FP32
    else:
        raise ValueError("dtype must be bfloat16 or float32")
    if not same or k.dtype is not dtype or k.device != dev or q.stride(-1) != 1 or k.stride(-1) != 1:
        raise ValueError("q and k must share type, device and all sizes but the heads, which must be contiguous")
    half = inv_freq.numel()
    _b._in(inv_freq, (half,), torch.float64, dev, "inv_freq")
    if q_weight is not None:
        _b._in(q_weight, (d,), dtype, dev, "q_weight")
    if k_weight is not None:
        _b._in(k_weight, (d,), dtype, dev, "k_weight")
    if ends is not None:
        _b._in(ends, (B,), torch.int32, dev, "ends")
    return B, N, Hq, Hkv, d, 2 * half, code, qs, ks, dtype, dev


def _out_like(t, shape, dtype, device, name, stream):
    """A caller-supplied output of rows of heads, or a new contiguous one."""
    if t is None:
        return _b._out(None, shape, dtype, device, name, stream)
    return _like(t, shape, dtype, device, name)


def qk_norm_rope(q, k, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                 cu_seqlens=None, ends=None, q_out=None, k_out=None, stream=None):
    """q_out, k_out = fa_qk_norm_rope(...): each head of q and k divided by its
    root mean square and multiplied by the weight ([d]; None leaves the norm
    out), its first 2 * len(inv_freq) elements then rotated by the token's
    position times inv_freq (float64).
    q [B, Hq, N, d] and k [B, Hkv, N, d], or packed [total, H, d] with
    cu_seqlens (int32 [B + 1]); bf16 or fp32, any strides with contiguous heads
    (views of a packed projection). The first token is at position 0, or the
    last at ends[b] - 1 (int32 [B]). q_out and k_out, of any such strides, may
    be q and k themselves. Returns (q_out, k_out)."""
    lib = _b.load()
    B, N, Hq, Hkv, d, rot, code, qs, ks, dtype, dev = _norm_sizes(q, k, inv_freq, q_weight, k_weight, cu_seqlens, ends)
    q_out = _out_like(q_out, qs, dtype, dev, "q_out", stream)
    k_out = _out_like(k_out, ks, dtype, dev, "k_out", stream)
    rc = lib.fa_qk_norm_rope(_rows(q), _rows(k), _rows(q_out), _rows(k_out), _b._ptr(q_weight), _b._ptr(k_weight),
                             float(eps), inv_freq.data_ptr(), rot, int(bool(interleaved)), _b._ptr(cu_seqlens),
                             _b._ptr(ends), B, N, Hq, Hkv, d, code, _b._stream_handle(stream))
    if rc != _b.FA_OK:
        raise _b.FAError(rc, "fa_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(q, k, dq_out, dk_out, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6,
                          interleaved: bool = False, cu_seqlens=None, ends=None, dq=None, dk=None, dq_weight=None,
                          dk_weight=None, ws=None, stream=None):
    """dq, dk, dq_weight, dk_weight = fa_qk_norm_rope_bwd(...): the gradients of
    qk_norm_rope's inputs and weights (float32 [d]; None where there is no
    weight) from those of its outputs. q and k are qk_norm_rope's inputs; dq
    and dk, of any strides with contiguous heads, may be dq_out and dk_out."""
    lib = _b.load()
    B, N, Hq, Hkv, d, rot, code, qs, ks, dtype, dev = _norm_sizes(q, k, inv_freq, q_weight, k_weight, cu_seqlens, ends)
    _like(dq_out, qs, dtype, dev, "dq_out")
    _like(dk_out, ks, dtype, dev, "dk_out")
    dq = _out_like(dq, qs, dtype, dev, "dq", stream)
    dk = _out_like(dk, ks, dtype, dev, "dk", stream)
    if q_weight is not None:
        dq_weight = _b._out(dq_weight, (d,), torch.float32, dev, "dq_weight", stream)
    elif dq_weight is not None:
        raise ValueError("dq_weight without a weight")
    if k_weight is not None:
        dk_weight = _b._out(dk_weight, (d,), torch.float32, dev, "dk_weight", stream)
    elif dk_weight is not None:
        raise ValueError("dk_weight without a weight")
    ws = _b._ws(ws, lambda: lib.fa_qk_norm_rope_bwd_workspace_size(d), dev, stream)
    rc = lib.fa_qk_norm_rope_bwd(_rows(q), _rows(k), _rows(dq_out), _rows(dk_out), _rows(dq), _rows(dk),
                                 _b._ptr(q_weight), _b._ptr(k_weight), _b._ptr(dq_weight), _b._ptr(dk_weight),
                                 float(eps), inv_freq.data_ptr(), rot, int(bool(interleaved)), _b._ptr(cu_seqlens),
                                 _b._ptr(ends), B, N, Hq, Hkv, d, code, ws.data_ptr(), _b._nbytes(ws),
                                 _b._stream_handle(stream))
    if rc != _b.FA_OK:
        raise _b.FAError(rc, "fa_qk_norm_rope_bwd")
    return dq, dk, dq_weight, dk_weight


def qk_norm_rope_append(q, k, v, k_cache, v_cache, k_scale, v_scale, slots, inv_freq, cu_seqlens, ends=None,
                        q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False, q_out=None,
                        stream=None):
    """q_out = fa_qk_norm_rope_append(...): qk_norm_rope of a serving step's
    packed new tokens with the keys, and v, stored into the cache as
    cache_append does. q [total, Hq, d], k, v [total, Hkv, d] bf16, any strides
    with contiguous heads; ends: the requests' lengths with the new tokens
    (cache_len behind cache_plan, a shared prefix added). Returns q_out [total,
    Hq, d]."""
    lib = _b.load()
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is needed")
    B, total, Hq, Hkv, d, rot, code, qs, ks, dtype, dev = _norm_sizes(q, k, inv_freq, q_weight, k_weight, cu_seqlens,
                                                                      ends)
    if code != _b.FA_BF16:
        raise ValueError("the cache takes bfloat16 inputs")
    _like(v, ks, dtype, dev, "v")
    num_blocks, H, bs, dc = _b._check_paged(k_cache, v_cache, k_scale, v_scale, dev)
    if H != Hkv or dc != d:
        raise ValueError("the cache must have k's heads")
    _b._in(slots, (total,), torch.int32, dev, "slots")
    q_out = _out_like(q_out, qs, dtype, dev, "q_out", stream)
    rc = lib.fa_qk_norm_rope_append(_rows(q), _rows(k), _rows(v), _rows(q_out), k_cache.data_ptr(), v_cache.data_ptr(),
                                    k_scale.data_ptr(), v_scale.data_ptr(), slots.data_ptr(), _b._ptr(q_weight),
                                    _b._ptr(k_weight), float(eps), inv_freq.data_ptr(), rot, int(bool(interleaved)),
                                    _b._ptr(cu_seqlens), _b._ptr(ends), B, total, Hq, Hkv, d, num_blocks, bs,
                                    _b._stream_handle(stream))
    if rc != _b.FA_OK:
        raise _b.FAError(rc, "fa_qk_norm_rope_append")
    return q_out


def qk_norm_rope_bwd_workspace_size(d) -> int:
    return _b.load().fa_qk_norm_rope_bwd_workspace_size(d)
