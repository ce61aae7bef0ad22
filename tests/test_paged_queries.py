"""GPU checks of fa_fwd_paged with infinities and NaN in Q: such a row has no
finite result, in either kernel and whatever K is there, and no other row is
touched; a row that sees no token stays zero whatever its query is."""

import numpy as np
import pytest

from oracle import paged as P
from test_paged import bf16, check, make_cache, run_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,old,G", [(1, 60, 4), (1, 9000, 4), (4, 200, 5), (40, 3000, 1), (40, 77, 4), (140, 60, 2),
                                     (140, 12000, 1)])
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("positive", [False, True])
def test_rows_without_a_finite_result(cuda_device, d, n, old, G, what, positive):
    """positive: K has one sign in the channel, so that every score of the row
    is the same infinity."""
    lens, cu = [old + n], [0, n]
    rng = np.random.default_rng(n + old)
    kb, vb, ks, vs, table = make_cache(lens, 64, 1, d, seed=n + d)
    if positive:
        kb[..., 7] = P.e4m3_encode(rng.uniform(1, 60, kb.shape[:-1]))
    q = rng.normal(size=(n, G, d))
    rows = q.reshape(n * G, d)
    wild = np.zeros(n * G, bool)
    wild[rng.permutation(n * G)[: max(1, n * G // 20)]] = True
    wild[-1] = True
    if n * G > 128:
        wild[[0, 127, 128]] = True
    if n * G == 1:
        wild[0] = True
    rows[wild, 7] = what
    q = rows.reshape(n, G, d)
    c = (kb, vb, ks, vs, table)
    o, lse = run_attend(bf16(q, cuda_device), c, cu, lens, n, True, cuda_device, 0.1)
    no = wild.reshape(n, G)
    assert np.isnan(o[no]).all() and np.isnan(lse.T[no]).all()
    assert np.isfinite(o[~no]).all() and np.isfinite(lse.T[~no]).all()
    if old <= 200:                                         # the others are what they are without them
        rows[wild] = 0
        zero = bf16(rows.reshape(n, G, d), cuda_device)
        ref = P.attend(zero.double().cpu().numpy(), *c[:4], cu, lens, table, 0.1)
        for a, r in ((o, ref[0]), (lse.T, ref[1].T)):
            a[no] = r[no]
        check(o, lse, ref, cu, G, slice(0, n), lens[0], d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,G", [(3, 2), (70, 3), (300, 1)])
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
def test_rows_that_see_nothing_stay_zero(cuda_device, d, n, G, what):
    lens, cu = [n - 2], [0, n]
    c = make_cache(lens, 16, 1, d, seed=n)
    q = np.random.default_rng(n).normal(size=(n, G, d))
    q[:2, :, 3] = what
    o, lse = run_attend(bf16(q, cuda_device), c, cu, lens, n, True, cuda_device, 0.1)
    assert (o[:2] == 0).all() and np.isneginf(lse[:, :2]).all()
    assert np.isfinite(o[2:]).all() and np.isfinite(lse[:, 2:]).all()
