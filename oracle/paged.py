"""fp64 oracle for the paged 8-bit key/value cache: the block plan, the
quantising append and attention over the cache, request by request and row by
row, as include/fa.h states them.

Test infrastructure only: imported by ``tests/``. The product path never uses
it.

E4M3 numbers are held as their bytes (uint8); :func:`e4m3_decode` and
:func:`e4m3_encode` are the format's definition (1 sign, 4 exponent bits with
bias 7, 3 fraction bits, no infinities, 0x7F and 0xFF are NaN, largest 448).
"""

from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
EXP_MIN = -126


def _table():
    t = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if e == 15 and f == 7:
            x = np.nan
        t[b] = -x if b & 128 else x
    return t


E4M3 = _table()


def e4m3_decode(b):
    return E4M3[np.asarray(b, dtype=np.uint8)]


def e4m3_encode(x):
    """Nearest E4M3 byte (ties to the even byte), saturating; NaN to 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    pos = E4M3[:127]                                   # 0 .. 448 ascending
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), E4M3_MAX)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)      # first number >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(pos[hi] == a, hi, code)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def plan(new_len, cache_len, block_table, free_blocks, free_state, block_size, total):
    """The lists after one plan: dict of cache_len, block_table, free_blocks,
    free_state, cu_seqlens, slots, and refused (for want of blocks)."""
    bs, table, ring = block_size, np.array(block_table), np.array(free_blocks)
    cap = len(ring)
    head, count = int(free_state[0]), int(free_state[1])
    asked = granted = 0
    lens, cu, slots, refused, freed = [], [0], [], [], []
    for b, (n, c) in enumerate(zip(np.asarray(new_len).tolist(), np.asarray(cache_len).tolist())):
        had = -(-c // bs)
        if n < 0:
            freed += table[b, :had].tolist()
            lens.append(0)
            cu.append(cu[-1])
            continue
        need = -(-(c + n) // bs) - had
        asked += need
        cu.append(cu[-1] + n)
        if need and asked > count:
            refused.append(b)
            lens.append(c)
            slots += [-1] * n
            continue
        for j in range(had, had + need):
            table[b, j] = free_blocks[(head + granted) % cap]
            granted += 1
        slots += [int(table[b, p // bs]) * bs + p % bs for p in range(c, c + n)]
        lens.append(c + n)
    for i, blk in enumerate(freed):
        ring[(head + count + i) % cap] = blk
    slots += [-1] * (total - len(slots))
    i32 = np.int32
    return dict(cache_len=np.array(lens, i32), block_table=table.astype(i32), free_blocks=ring.astype(i32),
                free_state=np.array([(head + granted) % cap, count - granted + len(freed)], i32),
                cu_seqlens=np.array(cu, i32), slots=np.array(slots, i32), refused=refused)


def scale_exponent(amax):
    """e with 2^e the scale of a run whose largest finite magnitude is amax."""
    if amax == 0:
        return EXP_MIN
    f, x = np.frexp(amax)                            # amax = f 2^x, 0.5 <= f < 1; 448 = 0.875 2^9
    return max(x - 9 + (1 if f > 0.875 else 0), EXP_MIN)


def append(x, cache, scale, slots):
    """New rows x [total, H, d] into (bytes [nb, H, bs, d], scale [nb, H]);
    returns the new (bytes, scale)."""
    x = np.asarray(x, dtype=np.float64)
    cache, scale = np.array(cache), np.array(scale, dtype=np.float64)
    nb, H, bs, _ = cache.shape
    slots = np.asarray(slots).tolist()
    t = 0
    while t < len(slots):
        if not 0 <= slots[t] < nb * bs:
            t += 1
            continue
        blk, first = divmod(slots[t], bs)
        u = t
        while u < len(slots) and 0 <= slots[u] < nb * bs and slots[u] // bs == blk:
            u += 1
        for h in range(H):
            run = x[t:u, h]
            fin = np.abs(run[np.isfinite(run)])
            s = 2.0 ** scale_exponent(fin.max() if fin.size else 0.0)
            old = scale[blk, h] if first > 0 else 0.0
            if old > 0:
                f, e = np.frexp(old)
                s = max(s, 2.0 ** (e - 1 if f == 0.5 else e))
            if first > 0 and s != old:
                cache[blk, h, :first] = e4m3_encode(e4m3_decode(cache[blk, h, :first]) * (old / s))
            for i in range(t, u):
                cache[blk, h, slots[i] % bs] = e4m3_encode(x[i, h] / s)
            scale[blk, h] = s
        t = u
    return cache, scale


def attend(q, k_bytes, v_bytes, k_scale, v_scale, cu_seqlens, cache_len, block_table, scale, causal=True):
    """O [total, Hq, d], L [Hq, total] and, for tolerances, the weighted
    absolute values A = sum_j P_j |v_j|, the score magnitudes
    X = max_j scale |q| . |k_j| of each row and their bound
    Y = max_j scale max|q| sum|k_j|."""
    q = np.asarray(q, dtype=np.float64)
    total, Hq, d = q.shape
    nb, Hkv, bs, _ = k_bytes.shape
    G = Hq // Hkv
    O, A = np.zeros((total, Hq, d)), np.zeros((total, Hq, d))
    L, X, Y = np.full((Hq, total), -np.inf), np.zeros((Hq, total)), np.zeros((Hq, total))
    for b in range(len(cache_len)):
        t0, n, length = int(cu_seqlens[b]), int(cu_seqlens[b + 1] - cu_seqlens[b]), int(cache_len[b])
        if n == 0 or length == 0:
            continue
        blocks = block_table[b, : -(-length // bs)]
        for h in range(Hkv):
            k = (e4m3_decode(k_bytes[blocks, h]) * np.asarray(k_scale, np.float64)[blocks, h][:, None, None])
            v = (e4m3_decode(v_bytes[blocks, h]) * np.asarray(v_scale, np.float64)[blocks, h][:, None, None])
            k, v = k.reshape(-1, d)[:length], v.reshape(-1, d)[:length]
            for i in range(n):
                seen = min(max(length - n + i + 1, 0), length) if causal else length
                if seen == 0:
                    continue
                for g in range(h * G, (h + 1) * G):
                    s = scale * (k[:seen] @ q[t0 + i, g])
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    O[t0 + i, g] = p @ v[:seen] / l
                    A[t0 + i, g] = p @ np.abs(v[:seen]) / l
                    L[g, t0 + i] = m + np.log(l) if l > 0 else np.nan
                    X[g, t0 + i] = (scale * (np.abs(k[:seen]) @ np.abs(q[t0 + i, g]))).max()
                    Y[g, t0 + i] = scale * np.abs(q[t0 + i, g]).max() * np.abs(k[:seen]).sum(1).max()
    return O, L, A, X, Y
