"""GPU checks of fa_fwd_paged's numerics where operands span many binary
orders: what one request's result is good for may not depend on which kernel
takes it."""

import math

import numpy as np
import pytest

from oracle import paged as P
from test_paged import bf16, make_cache, run_attend

pytestmark = pytest.mark.gpu


def close(o, lse, ref, visible, d, left=0.0):
    """Scores: d products and sums in fp32 (d 2^-24 of X = max sum |q k|), the
    scale factors and the exponent's argument (16 roundings of 2^-24 of it), and
    Q within 2^-31 of its row's largest value (2^-31 Y), or, where its elements
    are within 2^13 of one another, 2^-20 of it in all (left). Weights: f16 (2^-11),
    fp32 sums (2^-20), twice the score error, and 2^-31 of the largest for what
    vanishes. O: that on A = sum P |v|, and bf16 (2^-8 |O|)."""
    O, L, A, X, Y = ref
    ds = (d + 16) * 2.0 ** -24 * X + 2.0 ** -31 * Y + left
    empty = np.isneginf(L)
    assert np.array_equal(empty, np.isneginf(lse))
    with np.errstate(invalid="ignore"):
        el = np.where(empty, 0.0, np.abs(lse - L))
    tl = ds + 2.0 ** -18 + 2.0 ** -21 * np.abs(np.where(empty, 0.0, L))
    assert (el <= tl).all(), (el / tl).max()
    w = (2.0 ** -11 + 2.0 ** -20 + 2 * ds + visible * 2.0 ** -31).T[..., None]
    eo, to = np.abs(o - O), 2.0 ** -8 * np.abs(O) + w * A * 1.01 + 1e-30
    assert (eo <= to).all(), (eo / to).max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pairs", [[(300, 1)], [(77, 3)], [(200, 40)], [(0, 150)], [(90, 3), (40, 60)]])
@pytest.mark.parametrize("ratio", [6, 10, 12, 14, 17, 20, 23])
def test_a_large_channel_of_q(cuda_device, d, pairs, ratio):
    """One channel of Q is 2^ratio times the others, and K is zero there: the
    scores come from the small ones. In the last case three tokens of one
    request stand beside a prompt."""
    lens = [c + n for c, n in pairs]
    cu = np.concatenate([[0], np.cumsum([n for _, n in pairs])])
    rng = np.random.default_rng(ratio + d)
    kb, vb, ks, vs, table = make_cache(lens, 32, 1, d, seed=ratio)
    kb[..., 5] = 0
    q = rng.normal(size=(int(cu[-1]), 2, d))
    q[..., 5] = 2.0 ** ratio * rng.uniform(1, 2, q.shape[:2])
    q = bf16(q, cuda_device)
    scale = 1 / math.sqrt(d)
    o, lse = run_attend(q, (kb, vb, ks, vs, table), cu, lens, max(n for _, n in pairs), True, cuda_device, scale)
    qn = q.double().cpu().numpy()
    ref = P.attend(qn, kb, vb, ks, vs, cu, lens, table, scale)
    left = 2.0 ** -20 * scale * np.abs(qn).max(-1).T * 448 * ks.max() if ratio == 6 else 0.0
    close(o, lse, ref, max(lens), d, left)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 40, 140])
def test_channels_of_q_and_k_over_many_orders(cuda_device, d, n):
    """Every channel of Q has a magnitude of its own, over sixteen binary
    orders, and K the opposite one, as far as its format reaches."""
    lens, cu = [n + 130], [0, n]
    rng = np.random.default_rng(n + d)
    e = rng.integers(-8, 9, d)
    kb, vb, ks, vs, table = make_cache(lens, 16, 1, d, seed=n)
    kb = P.e4m3_encode(np.clip(rng.normal(size=kb.shape) * 2.0 ** np.clip(-e, -6, 6), -448, 448))
    q = bf16(rng.normal(size=(n, 3, d)) * 2.0 ** e, cuda_device)
    ks[:] = 2.0 ** -2
    o, lse = run_attend(q, (kb, vb, ks, vs, table), cu, lens, n, True, cuda_device, 0.1)
    ref = P.attend(q.double().cpu().numpy(), kb, vb, ks, vs, cu, lens, table, 0.1)
    close(o, lse, ref, max(lens), d)
