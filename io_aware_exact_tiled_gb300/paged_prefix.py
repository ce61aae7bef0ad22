"""Binding of attention over the paged cache with shared prefixes
(fa_fwd_paged_prefix of include/fa.h), as binding.py binds the other calls."""

from __future__ import annotations

import math
from typing import Optional

import torch

from . import binding as _b


def fwd_paged_prefix_workspace_size(B, P, Hq, Hkv, total, max_new, d) -> int:
    return _b.load().fa_fwd_paged_prefix_workspace_size(B, P, Hq, Hkv, total, max_new, d)


def forward_paged_prefix(q, k_cache, v_cache, k_scale, v_scale, cu_seqlens, cache_len, block_table, prefix_cu,
                         prefix_len, prefix_table, max_new: int, scale: Optional[float] = None, causal: bool = True,
                         out=None, lse=None, ws=None, stream=None):
    """O, L = fa_fwd_paged_prefix(...): forward_paged for groups of requests
    that share a prefix of the cache. Group p is requests prefix_cu[p] ..
    prefix_cu[p + 1] - 1 (int32 [P + 1]); its prefix is prefix_len[p] tokens
    (int32 [P]) in the blocks prefix_table[p] (int32 [P, max_prefix_blocks]).
    cache_len and block_table are the requests' own tokens. Returns (o [total,
    Hq, d], lse fp32 [Hq, total])."""
    lib = _b.load()
    _b._check_device(q)
    dev = q.device
    num_blocks, Hkv, bs, d = _b._check_paged(k_cache, v_cache, k_scale, v_scale, dev)
    if q.dim() != 3 or block_table.dim() != 2 or cache_len.dim() != 1 or prefix_table.dim() != 2:
        raise ValueError("expected q [total, Hq, d], block_table [B, max_blocks], cache_len [B] and prefix_table"
                         " [P, max_prefix_blocks]")
    total, Hq, _ = q.shape
    B, max_blocks = block_table.shape
    P, max_prefix = prefix_table.shape
    i32 = torch.int32
    _b._in(q, (total, Hq, d), torch.bfloat16, dev, "q")
    _b._in(cu_seqlens, (B + 1,), i32, dev, "cu_seqlens")
    _b._in(cache_len, (B,), i32, dev, "cache_len")
    _b._in(block_table, (B, max_blocks), i32, dev, "block_table")
    _b._in(prefix_cu, (P + 1,), i32, dev, "prefix_cu")
    _b._in(prefix_len, (P,), i32, dev, "prefix_len")
    _b._in(prefix_table, (P, max_prefix), i32, dev, "prefix_table")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = _b._out(out, q.shape, q.dtype, dev, "out", stream)
    L = _b._out(lse, (Hq, total), torch.float32, dev, "lse", stream)
    ws = _b._ws(ws, lambda: lib.fa_fwd_paged_prefix_workspace_size(B, P, Hq, Hkv, total, int(max_new), d), dev,
             stream)
    rc = lib.fa_fwd_paged_prefix(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                                 v_scale.data_ptr(), o.data_ptr(), L.data_ptr(), cu_seqlens.data_ptr(),
                                 cache_len.data_ptr(), block_table.data_ptr(), prefix_cu.data_ptr(),
                                 prefix_len.data_ptr(), prefix_table.data_ptr(), B, P, Hq, Hkv, total, int(max_new),
                                 max_blocks, max_prefix, num_blocks, bs, d, scale, int(bool(causal)), ws.data_ptr(),
                                 _b._nbytes(ws), _b._stream_handle(stream))
    if rc != _b.FA_OK:
        raise _b.FAError(rc, "fa_fwd_paged_prefix")
    return o, L
