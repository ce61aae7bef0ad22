"""GPU checks of what the kernels of fa_fwd_paged reuse while they run: the
row-tile kernel over many short pieces, whose row tiles without rows or keys
fall behind the roles that feed them, and the rings of the split-key kernel."""

import math

import numpy as np
import pytest
import torch

import io_aware_exact_tiled_gb300 as fa
from oracle import paged as P
from test_paged import bf16, check, make_cache, run_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_a_long_cut_unit_in_front_of_many_short_ones(cuda_device, d):
    """One request of 40 rows over a long cache, cut over many CTAs, then
    hundreds of requests of 33 to 200 rows (the second row tile without rows,
    or with a few), NaN values in the last token of some. The same bits each
    time, and within the bounds; a NaN reaches the row that sees it only."""
    rng = np.random.default_rng(d)
    n = np.concatenate([[40], rng.integers(33, 201, 300)])
    n[1:200:2] = rng.integers(33, 128, 100)
    lens = n + np.concatenate([[30000], rng.integers(0, 90, 300)])
    cu = np.concatenate([[0], np.cumsum(n)])
    total, scale = int(cu[-1]), 1 / math.sqrt(d)
    kb, vb, ks, vs, table = make_cache(lens.tolist(), 64, 1, d, seed=d)
    q = bf16(rng.normal(size=(total, 1, d)), cuda_device)
    O, L, A, X, Y = P.attend(q.double().cpu().numpy(), kb, vb, ks, vs, cu, lens, table, scale)
    nan = np.zeros((total, d), bool)
    for b in range(1, 301, 3):
        pos, col = int(lens[b]) - 1, b % d
        vb[table[b, pos // 64], 0, pos % 64, col] = 0x7F
        nan[cu[b + 1] - 1, col] = True
    c = (kb, vb, ks, vs, table)
    o, lse = run_attend(q, c, cu, lens.tolist(), int(n.max()), True, cuda_device, scale)
    for _ in range(10):
        again = run_attend(q, c, cu, lens.tolist(), int(n.max()), True, cuda_device, scale)
        np.testing.assert_array_equal(o, again[0])
        np.testing.assert_array_equal(lse, again[1])
    np.testing.assert_array_equal(np.isnan(o[:, 0]), nan)
    # the columns with a NaN in them count as right, the others of their rows are checked
    o[:, 0][nan] = O[:, 0][nan]
    check(o, lse, (O, L, A, X, Y), cu, 1, slice(0, total), int(lens.max()), d)


@pytest.mark.parametrize("d,G,Hkv", [(64, 1, 2), (64, 8, 1), (128, 2, 2), (128, 8, 1)])
def test_many_row_tiles_that_see_nothing(cuda_device, d, G, Hkv):
    """Requests of thousands of new tokens of which only the last few are
    cached: one unit after the other has a row tile, or both, without keys."""
    n, lens = [3000, 70, 2500], [10, 300, 141]
    cu = np.concatenate([[0], np.cumsum(n)])
    total = int(cu[-1])
    rng = np.random.default_rng(d + G)
    c = make_cache(lens, 16, Hkv, d, seed=G)
    q = bf16(rng.normal(size=(total, Hkv * G, d)), cuda_device)
    ref = P.attend(q.double().cpu().numpy(), *c[:4], cu, lens, c[4], 0.1)
    for _ in range(5):
        o, lse = run_attend(q, c, cu, lens, max(n), True, cuda_device, 0.1)
        check(o, lse, ref, cu, G, slice(0, total), max(lens), d)
    assert torch.isfinite(torch.from_numpy(o)).all()


@pytest.mark.parametrize("d,G,n", [(64, 4, 1), (64, 4, 3), (64, 8, 4), (128, 4, 1), (128, 7, 2), (128, 8, 3)])
@pytest.mark.parametrize("bs", [16, 64])
def test_split_key_rings_again_and_again(cuda_device, d, G, n, bs):
    """The split-key kernel's rings turn over thousands of times while another
    stream keeps the memory busy: the same bits each time, and within the
    bounds (long requests, cut, and short ones, a warp each)."""
    rng = np.random.default_rng(d + G + n)
    for lens in ([9000, 40, 5000, 17, 2500], rng.integers(n, 300, 400).tolist()):
        cu = n * np.arange(len(lens) + 1)
        total = int(cu[-1])
        c = make_cache(lens, bs, 2, d, seed=bs)
        q = bf16(rng.normal(size=(total, 2 * G, d)), cuda_device)
        ref = P.attend(q.double().cpu().numpy(), *c[:4], cu, lens, c[4], 0.1)
        o, lse = run_attend(q, c, cu, lens, n, True, cuda_device, 0.1)
        check(o, lse, ref, cu, G, slice(0, total), max(lens), d)
        kb, vb, ks, vs, table = c
        args = [torch.tensor(x, device=cuda_device).view(torch.float8_e4m3fn) for x in (kb, vb)]
        args += [torch.tensor(x, device=cuda_device) for x in (ks, vs)]
        args += [torch.tensor(np.asarray(x), dtype=torch.int32, device=cuda_device) for x in (cu, lens, table)]
        side, busy = torch.cuda.Stream(), torch.empty(1 << 26, device=cuda_device)
        side.wait_stream(torch.cuda.current_stream())
        first = fa.forward_paged(q, *args, n, scale=0.1)
        for i in range(60):
            if i % 3 == 0:
                with torch.cuda.stream(side):
                    busy.add_(1.0)
            again = fa.forward_paged(q, *args, n, scale=0.1)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1]), i
        torch.cuda.synchronize()
        np.testing.assert_array_equal(first[0].double().cpu().numpy(), o)
