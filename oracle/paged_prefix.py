"""fp64 oracle for attention over the paged cache with shared prefixes: each
request's keys are its group's prefix and then its own tokens.

Test infrastructure only: imported by ``tests/``. The product path never uses
it.
"""

from __future__ import annotations

import numpy as np

from .paged import e4m3_decode


def _rows(cache, scale, table, length, h, bs):
    at = np.asarray(table)[: -(-length // bs)]
    x = e4m3_decode(cache[at, h]) * np.asarray(scale, np.float64)[at, h][:, None, None]
    return x.reshape(-1, cache.shape[-1])[:length]


def attend(q, k_bytes, v_bytes, k_scale, v_scale, cu_seqlens, cache_len, block_table, prefix_cu, prefix_len,
           prefix_table, scale, causal=True):
    """O, L, A, X and Y as oracle.paged.attend returns them."""
    q = np.asarray(q, dtype=np.float64)
    total, Hq, d = q.shape
    _, Hkv, bs, _ = k_bytes.shape
    G = Hq // Hkv
    O, A = np.zeros((total, Hq, d)), np.zeros((total, Hq, d))
    L, X, Y = np.full((Hq, total), -np.inf), np.zeros((Hq, total)), np.zeros((Hq, total))
    for b in range(len(cache_len)):
        t0, n, length = int(cu_seqlens[b]), int(cu_seqlens[b + 1] - cu_seqlens[b]), int(cache_len[b])
        group = [p for p in range(len(prefix_len)) if prefix_cu[p] <= b < prefix_cu[p + 1]]
        before = int(prefix_len[group[0]]) if group else 0
        for h in range(Hkv if n else 0):
            parts = [_rows(c, s, block_table[b], length, h, bs) for c, s in ((k_bytes, k_scale), (v_bytes, v_scale))]
            if before:
                parts = [np.concatenate([_rows(c, s, prefix_table[group[0]], before, h, bs), x])
                         for (c, s), x in zip(((k_bytes, k_scale), (v_bytes, v_scale)), parts)]
            k, v = parts
            for i in range(n):
                seen = before + (min(max(length - n + i + 1, 0), length) if causal else length)
                if seen == 0:
                    continue
                for y in range(h * G, (h + 1) * G):
                    s = scale * (k[:seen] @ q[t0 + i, y])
                    m = s.max()
                    p = np.exp(s - m)
                    O[t0 + i, y] = p @ v[:seen] / p.sum()
                    A[t0 + i, y] = p @ np.abs(v[:seen]) / p.sum()
                    L[y, t0 + i] = m + np.log(p.sum())
                    X[y, t0 + i] = (scale * (np.abs(k[:seen]) @ np.abs(q[t0 + i, y]))).max()
                    Y[y, t0 + i] = scale * np.abs(q[t0 + i, y]).max() * np.abs(k[:seen]).sum(1).max()
    return O, L, A, X, Y
