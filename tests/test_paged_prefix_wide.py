"""GPU checks of units of one row tile in attention over shared prefixes: many
of them a CTA, queries of wide range among narrow ones, long prefixes; against
the fp64 oracle, and the same bits each time."""

import numpy as np
import pytest
import torch

from oracle import paged_prefix as PP

from test_paged_prefix import Batch

pytestmark = pytest.mark.gpu


def check(b, got):
    """As test_paged_precision states for queries of wide range (Q within 2^-31
    of its row's largest value, 2^-31 Y), with the joining of two parts (2^-19);
    of other rows 2^-20 of the largest value may be left out in all."""
    O, L, A, X, Y = PP.attend(b.q.double().cpu().numpy(), *b.c, b.cu, b.lens, b.table, b.pcu, b.plen, b.ptable, b.scale)
    o, lse = (x.double().cpu().numpy() for x in got)
    top = np.abs(b.q.double().cpu().numpy()).max(-1).T
    ds = (b.d + 16) * 2.0 ** -24 * X + 2.0 ** -31 * Y
    ds += np.where(top < 100, 2.0 ** -20 * b.scale * top * 448 * b.c[2].max(), 0.0)
    el, tl = np.abs(lse - L), ds + 2.0 ** -18 + 2.0 ** -21 * np.abs(L)
    assert (el <= tl).all(), (el / tl).max()
    seen = max(b.lens) + max(b.plen)
    w = (2.0 ** -11 + 2.0 ** -19 + 2 * ds + seen * 2.0 ** -31).T[..., None]
    eo, to = np.abs(o - O), 2.0 ** -8 * np.abs(O) + w * A * 1.01 + 1e-30
    assert (eo <= to).all(), (eo / to).max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P,each,Hkv,prefix", [(60, 6, 8, 300), (24, 15, 8, 700), (45, 9, 8, 150), (100, 2, 8, 128)])
def test_queries_of_wide_range_in_many_units(cuda_device, P, each, Hkv, prefix, d):
    """Units of several key tiles, more than there are CTAs, most of them whole in
    one. In two groups of three, one channel of some queries is 2^14 times larger and K
    is zero there, so that the scores come from what is small beside it."""
    pairs = [(i % 3, 1) for i in range(P * each)]
    b = Batch(pairs, [(p * each, prefix + 37 * (p % 5)) for p in range(P)], 32, Hkv, 8, d, cuda_device, seed=P, pad=0)
    b.c[0][..., 5] = 0
    q = b.q.clone()
    for t in range(len(pairs)):
        if t // each % 3 and (t % each == 0 or t % 4 == 1):
            q[t, ::3, 5] *= 2.0 ** 14
    b.q = q
    got = b.run()
    check(b, got)
    for _ in range(20):
        again = b.run()
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P,each,Hkv,prefix", [(1, 12, 2, 20000), (76, 1, 4, 2500), (9, 8, 4, 6000)])
def test_many_key_tiles_of_one_row_tile(cuda_device, P, each, Hkv, prefix, d):
    """Prefixes whose blocks lie anywhere: one cut over every CTA, and many of
    twenty and more key tiles in a CTA."""
    b = Batch([(i % 9, 1) for i in range(P * each)], [(p * each, prefix + p) for p in range(P)], 16, Hkv, 8, d,
              cuda_device, seed=P, pad=0)
    got = b.run()
    b.check(got=got)
    for _ in range(20):
        again = b.run()
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
