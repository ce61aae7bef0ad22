"""Pins of the paged-cache oracle (CPU): the E4M3 tables against torch's
float8 type, the plan against its invariants, the append against closed forms,
attention against the contiguous decoding oracle."""

import numpy as np
import torch

from oracle import decode as DEC
from oracle import paged as P


def test_e4m3_decode_matches_torch():
    b = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(P.e4m3_decode(b.numpy()), b.view(torch.float8_e4m3fn).double().numpy())


def test_e4m3_encode_matches_torch_and_rounds_ties_to_even():
    pos = P.E4M3[:127]
    mids = (pos[1:] + pos[:-1]) / 2
    x = np.concatenate([pos, mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9),
                        np.random.default_rng(0).normal(0, 60, 4000)])
    x = x[np.abs(x) <= 448]
    x32 = x.astype(np.float32)
    want = torch.from_numpy(x32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(P.e4m3_encode(x32), want)
    np.testing.assert_array_equal(P.e4m3_encode(-x32[x32 > 0]), want[x32 > 0] | 128)
    np.testing.assert_array_equal(P.e4m3_encode([1e9, -np.inf, np.nan, 449.0]), [126, 254, 127, 126])


def test_scale_exponent_is_the_least_that_fits():
    for amax in (448.0, 448.0000001, 1.0, 0.875, 0.88, 1e-30, 3e38, 224.0, 225.0):
        e = P.scale_exponent(amax)
        assert amax <= 448 * 2.0 ** e and (amax > 448 * 2.0 ** (e - 1) or e == P.EXP_MIN)
    assert P.scale_exponent(0.0) == P.scale_exponent(1e-40) == -126


def test_plan_hands_out_every_block_once_and_takes_them_back():
    rng = np.random.default_rng(1)
    nb, bs, B, mb = 40, 16, 7, 12
    s = dict(cache_len=np.zeros(B, np.int32), block_table=np.full((B, mb), -1, np.int32),
             free_blocks=rng.permutation(nb).astype(np.int32), free_state=np.array([33, nb], np.int32))
    for _ in range(200):
        new = rng.integers(-1, 40, B)
        new = np.where(s["cache_len"] + new > mb * bs, -1, new)
        total = int(new.clip(0).sum()) + 3
        r = P.plan(new, s["cache_len"], s["block_table"], s["free_blocks"], s["free_state"], bs, total)
        used = [blk for b in range(B) for blk in r["block_table"][b, : -(-int(r["cache_len"][b]) // bs)]]
        head, count = r["free_state"]
        free = [r["free_blocks"][(head + i) % nb] for i in range(count)]
        assert sorted(used + free) == list(range(nb))
        live = r["slots"][r["slots"] >= 0]
        assert len(set(live.tolist())) == len(live) and (r["slots"][total - 3:] == -1).all()
        for b in range(B):
            if b in r["refused"]:
                assert r["cache_len"][b] == s["cache_len"][b]
        s = {k: r[k] for k in s}


def test_append_closed_forms():
    nb, H, bs, d = 3, 2, 16, 64
    cache, scale = np.zeros((nb, H, bs, d), np.uint8), np.zeros((nb, H))
    x = np.full((2, H, d), 1.0)
    x[:, 1] = 448.0
    c, s = P.append(x, cache, scale, [16, 17])
    assert s[1, 0] == 2.0 ** -8 and s[1, 1] == 1.0 and (s[[0, 2]] == 0).all()
    assert (P.e4m3_decode(c[1, 0, :2]) == 256.0).all() and (P.e4m3_decode(c[1, 1, :2]) == 448.0).all()
    c2, s2 = P.append(np.full((1, H, d), 900.0), c, s, [18])       # the scales grow; old rows follow
    assert (s2[1] == 4.0).all()                                    # 900 / 448 = 2.009
    assert (P.e4m3_decode(c2[1, 0, :2]) * s2[1, 0] == 1.0).all()
    assert (P.e4m3_decode(c2[1, 1, :2]) * s2[1, 1] == 448.0).all()
    c3, s3 = P.append(np.full((1, H, d), 1.0), c2, s2, [16])       # row 0 starts the block anew
    assert (s3[1] == 2.0 ** -8).all() and (c3[1, :, 1:] == c2[1, :, 1:]).all()
    c4, s4 = P.append(x, c, s, [-1, nb * bs])                      # slots out of range
    assert (c4 == c).all() and (s4 == s).all()


def test_attend_equals_contiguous_decoding():
    rng = np.random.default_rng(3)
    nb, Hkv, bs, d, G = 9, 2, 16, 64, 3
    kb, vb = (rng.integers(0, 127, (nb, Hkv, bs, d)).astype(np.uint8) for _ in range(2))
    ks, vs = rng.uniform(0.001, 0.01, (nb, Hkv)), rng.uniform(0.001, 0.01, (nb, Hkv))
    table = np.array([[4, 0, 7], [2, 5, 8]])
    lens, n = [37, 48], 1
    q = rng.normal(size=(2, Hkv * G, d))
    O, L, *_ = P.attend(q, kb, vb, ks, vs, [0, 1, 2], lens, table, 0.125)
    k = (P.e4m3_decode(kb) * ks[..., None, None])[table].transpose(0, 2, 1, 3, 4).reshape(2, Hkv, -1, d)
    v = (P.e4m3_decode(vb) * vs[..., None, None])[table].transpose(0, 2, 1, 3, 4).reshape(2, Hkv, -1, d)
    k, v = np.repeat(k, G, 1), np.repeat(v, G, 1)
    Or, Lr = DEC.decode_forward(q[:, :, None], k, v, 0.125, np.array(lens))
    np.testing.assert_allclose(O, Or[:, :, 0], rtol=1e-12)
    np.testing.assert_allclose(L.T, Lr[:, :, 0], rtol=1e-12)


def test_attend_causal_rows_see_their_prefix():
    rng = np.random.default_rng(4)
    kb, vb = (rng.integers(0, 127, (2, 1, 16, 64)).astype(np.uint8) for _ in range(2))
    one = np.full((2, 1), 0.004)
    q = rng.normal(size=(5, 2, 64))
    table = np.array([[1, 0]])
    O, L, *_ = P.attend(q, kb, vb, one, one, [0, 5], [20], table, 0.1)
    for i in range(5):
        Oi, Li, *_ = P.attend(q[i:i + 1], kb, vb, one, one, [0, 1], [16 + i], table, 0.1, causal=False)
        np.testing.assert_allclose(O[i], Oi[0], rtol=1e-13)
        np.testing.assert_allclose(L[:, i], Li[:, 0], rtol=1e-13)
    O, L, *_ = P.attend(q, kb, vb, one, one, [0, 5], [3], table, 0.1)   # two rows before the first token
    assert (O[:2] == 0).all() and np.isneginf(L[:, :2]).all() and np.isfinite(L[:, 2:]).all()
