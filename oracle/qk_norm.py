"""fp64 oracle for the norm of queries and keys with rotation and its gradient,
head by head, as include/fa.h states them.

Test infrastructure only: imported by ``tests/``. The product path never uses
it. Angles are reduced to a fraction of a turn in whole numbers, exactly.
"""

from __future__ import annotations

import numpy as np

BITS = 220


def _arctan_inverse(n):
    """arctan(1 / n) as a multiple of 2^-(BITS + 20), by its series."""
    term = (1 << (BITS + 20)) // n
    total, k = 0, 1
    while term:
        total += term // k if k % 4 == 1 else -(term // k)
        term //= n * n
        k += 2
    return total


PI = (16 * _arctan_inverse(5) - 4 * _arctan_inverse(239)) >> 20   # Machin's formula, times 2^BITS
TURNS_PER_RADIAN = (1 << (2 * BITS)) // (2 * PI)                  # 1 / (2 pi), times 2^BITS


def angles(pos, inv_freq):
    """[tokens, rot / 2] angles in (-pi, pi], equal to pos * inv_freq modulo 2 pi."""
    out = np.empty((len(pos), len(inv_freq)))
    ratios = [float(f).as_integer_ratio() for f in inv_freq]
    for t, p in enumerate(pos):
        for i, (a, b) in enumerate(ratios):
            turn = int(p) * a * TURNS_PER_RADIAN // b % (1 << BITS)
            if turn > 1 << (BITS - 1):
                turn -= 1 << BITS
            out[t, i] = 2 * np.pi * (turn / (1 << BITS))
    return out


def positions(N, cu_seqlens=None, ends=None):
    """Position of each of N tokens and whether it is of a sequence."""
    pos, there = np.zeros(N, np.int64), np.zeros(N, bool)
    if cu_seqlens is None:
        return np.arange(N) + (0 if ends is None else int(ends) - N), ~there
    for b, (a, z) in enumerate(zip(cu_seqlens[:-1], cu_seqlens[1:])):
        pos[a:z] = np.arange(z - a) + (0 if ends is None else int(ends[b]) - (z - a))
        there[a:z] = True
    return pos, there


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _turn(y, a, u, v):
    """y [tokens, H, d] with pairs (u, v) turned by angles a, and the sums of
    the magnitudes that went into each element."""
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    z, m = y.copy(), np.abs(y)
    z[..., u] = y[..., u] * c - y[..., v] * s
    z[..., v] = y[..., u] * s + y[..., v] * c
    m[..., u] = m[..., v] = m[..., u] + m[..., v]
    return z, m


def forward(x, pos, weight, eps, inv_freq, interleaved):
    """z and, for tolerances, the magnitudes that each element is made of."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return _turn(x, angles(pos, inv_freq), *_pairs(2 * len(inv_freq), interleaved))


def backward(x, dz, pos, weight, eps, inv_freq, interleaved):
    """dx, dweight (None without a weight) and their magnitudes."""
    dz = np.asarray(dz, np.float64)
    u, m = _turn(dz, -angles(pos, inv_freq), *_pairs(2 * len(inv_freq), interleaved))
    if weight is None:
        return u, None, m, None
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    dx = r * (u * w - xh * (u * w * xh).mean(-1, keepdims=True))
    mx = r * (m * abs(w) + abs(xh) * (m * abs(w * xh)).mean(-1, keepdims=True))
    return dx, (u * xh).sum((0, 1)), mx, (m * abs(xh)).sum((0, 1))
