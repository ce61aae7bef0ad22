"""GPU checks of the paged 8-bit cache (fa_cache_plan, fa_cache_append,
fa_fwd_paged) against the fp64 oracle. The plan and the append have to be
equal; attention has to be within bounds counted from its roundings."""

import math

import numpy as np
import pytest
import torch

import io_aware_exact_tiled_gb300 as fa
from io_aware_exact_tiled_gb300 import binding as fb
from oracle import paged as P

pytestmark = pytest.mark.gpu


def dev_i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


# --------------------------------------------------------------------------
# plan
# --------------------------------------------------------------------------

PLAN_KEYS = ("cache_len", "block_table", "free_blocks", "free_state", "cu_seqlens", "slots")


def make_plan(B, bs, len_hi, new_hi, release, room, seed):
    """Numpy inputs of a plan: requests with blocks in an arbitrary order."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, len_hi + 1, B)
    n = rng.integers(0, new_hi + 1, B)
    n[rng.random(B) < release] = -1
    had = -(-c // bs)
    need = np.maximum(-(-(c + n.clip(0)) // bs) - had, 0)
    mb = max(1, int((had + need).max()))
    count = int(need.sum() * room)
    nb = max(1, int(had.sum()) + count + 3)
    perm = rng.permutation(nb)
    table = np.full((B, mb), -1)
    at = 0
    for b in range(B):
        table[b, :had[b]] = perm[at:at + had[b]]
        at += had[b]
    head = int(rng.integers(0, nb))
    ring = np.full(nb, -1)
    ring[(head + np.arange(count)) % nb] = perm[at:at + count]
    total = int(n.clip(0).sum()) + int(rng.integers(0, 4))
    return dict(new_len=n, cache_len=c, block_table=table, free_blocks=ring, free_state=np.array([head, count]),
                block_size=bs, total=total)


def run_plan(x, dev, in_place=False):
    t = {k: dev_i32(x[k], dev) for k in ("new_len", "cache_len", "block_table", "free_blocks", "free_state")}
    ws = fa.workspace(256, dev)
    out = {} if in_place else dict(cache_len_out=torch.full_like(t["cache_len"], 77),
                                   free_state_out=torch.full_like(t["free_state"], 77))
    cu, slots = fa.cache_plan(t["new_len"], t["cache_len"], t["block_table"], t["free_blocks"], t["free_state"],
                              x["block_size"], total=x["total"], ws=ws, **out)
    status = fa.get_status(ws)
    got = dict(cache_len=out.get("cache_len_out", t["cache_len"]), block_table=t["block_table"],
               free_blocks=t["free_blocks"], free_state=out.get("free_state_out", t["free_state"]),
               cu_seqlens=cu, slots=slots)
    if not in_place:
        np.testing.assert_array_equal(t["cache_len"].cpu().numpy(), x["cache_len"])
        np.testing.assert_array_equal(t["free_state"].cpu().numpy(), x["free_state"])
    return {k: v.cpu().numpy() for k, v in got.items()}, status


@pytest.mark.parametrize("B,bs,len_hi,new_hi,release,room", [
    (1, 64, 0, 1, 0.0, 1.0), (1, 16, 0, 5000, 0.0, 1.0), (3, 16, 40, 1, 0.0, 1.0), (16, 64, 900, 1, 0.2, 1.0),
    (17, 256, 3000, 700, 0.1, 0.5), (255, 32, 100, 33, 0.3, 0.9), (257, 128, 2000, 3, 0.0, 0.0),
    (1000, 16, 500, 2, 0.5, 0.97), (1025, 64, 500, 9, 0.1, 0.9), (5000, 16, 64, 40, 0.2, 0.6),
    (16384, 16, 20, 2, 0.1, 0.99), (2, 64, 70, 40000, 0.0, 1.0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_equals_the_definition(cuda_device, B, bs, len_hi, new_hi, release, room, in_place):
    x = make_plan(B, bs, len_hi, new_hi, release, room, seed=B + bs)
    want = P.plan(**x)
    got, status = run_plan(x, cuda_device, in_place)
    for k in PLAN_KEYS:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    assert status == (fb.FA_ERR_NO_BLOCKS if want["refused"] else fb.FA_OK)


def test_plan_only_releases(cuda_device):
    x = make_plan(9, 16, 100, 0, 1.0, 1.0, seed=3)
    x["total"] = 0
    got, status = run_plan(x, cuda_device)
    want = P.plan(**x)
    for k in PLAN_KEYS:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    assert status == fb.FA_OK and got["slots"].size == 0


@pytest.mark.parametrize("B", [6, 1500])
def test_plan_reports_what_does_not_fit(cuda_device, B):
    def run(**kw):
        x = make_plan(B, 16, 60, 20, 0.0, 1.0, seed=5)
        x["cache_len"][2] = 33
        x["new_len"][2] = 5
        x["block_table"][2, :3] = x["block_table"][2, :1]
        for k, v in kw.items():
            v(x[k]) if callable(v) else x.update({k: v})
        return x, *run_plan(x, cuda_device)

    def put(i, v):
        return lambda a: a.__setitem__(i, v)

    x, got, st = run(cache_len=put(2, -5))
    assert st == fb.FA_ERR_INVALID_ARG
    x, got, st = run(new_len=put(2, 1 << 30))              # longer than the table
    assert st == fb.FA_ERR_INVALID_ARG and got["cache_len"][2] == 33
    x, got, st = run(block_table=put((2, 2), 1 << 20))     # a table entry that is no block
    assert st == fb.FA_ERR_INVALID_ARG
    t0 = got["cu_seqlens"][2]
    assert (got["slots"][t0:t0 + 5] == -1).all()
    x, got, st = run(total=10)                             # a slot array that is too short
    assert st == fb.FA_ERR_INVALID_ARG and got["cu_seqlens"].max() == 10
    x, got, st = run(free_state=put(1, 1 << 20))
    assert st == fb.FA_ERR_INVALID_ARG
    x, got, st = run(free_state=put(0, -1))
    assert st == fb.FA_ERR_INVALID_ARG
    x, got, st = run(free_blocks=lambda a: a.fill(-7))     # ring entries that are no blocks
    assert st == fb.FA_ERR_INVALID_ARG and got["slots"].max() < len(x["free_blocks"]) * 16


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------

def bf16(x, dev):
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).to(dev)


def run_append(k, v, kb, vb, ks, vs, slots, dev):
    t = [torch.tensor(x, device=dev).view(torch.float8_e4m3fn) for x in (kb, vb)]
    s = [torch.tensor(x, dtype=torch.float32, device=dev) for x in (ks, vs)]
    fa.cache_append(k, v, *t, *s, dev_i32(slots, dev))
    return [x.view(torch.uint8).cpu().numpy() for x in t] + [x.cpu().numpy() for x in s]


def same_bytes(a, b):
    """E4M3 bytes, with the two NaN codes taken as one."""
    nan = lambda x: np.where((x & 127) == 127, 127, x)  # noqa: E731
    np.testing.assert_array_equal(nan(a), nan(b))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 64, 256])
@pytest.mark.parametrize("H,runs", [
    (1, [(0, 1)]), (2, [(3, 1), (0, 1), (15, 1), (7, 1)]), (3, [(0, 16), (5, 11), (0, 3)]), (2, [(1, 15)]),
    (5, [(0, 16)] * 9 + [(2, 1)] * 40)])
def test_append_equals_the_definition(cuda_device, d, bs, H, runs):
    """Each run: (row of its first token, tokens) within a block, scaled up to
    the block size; values over many magnitudes."""
    rng = np.random.default_rng(bs + d + len(runs))
    nb = len(runs) + 3
    f = bs // 16
    blocks = rng.permutation(nb)[: len(runs)]
    slots = np.concatenate([blk * bs + r * f + np.arange(n if n == 1 else n * f)
                            for blk, (r, n) in zip(blocks, runs)])
    total = len(slots)
    kb, vb = (rng.integers(0, 127, (nb, H, bs, d)).astype(np.uint8) | (rng.integers(0, 2, (nb, H, bs, d)) << 7)
              .astype(np.uint8) for _ in range(2))
    ks, vs = (2.0 ** rng.integers(-12, 3, (nb, H)) for _ in range(2))
    k, v = (rng.normal(size=(total, H, d)) * 2.0 ** rng.integers(-9, 9, (total, H, 1)) for _ in range(2))
    kt, vt = bf16(k, cuda_device), bf16(v, cuda_device)
    got = run_append(kt, vt, kb, vb, ks, vs, slots, cuda_device)
    for x, b0, s0, gb, gs in ((kt, kb, ks, got[0], got[2]), (vt, vb, vs, got[1], got[3])):
        wb, ws = P.append(x.double().cpu().numpy(), b0, s0, slots)
        np.testing.assert_array_equal(gs, ws.astype(np.float32))
        same_bytes(gb, wb)


@pytest.mark.parametrize("d,bs,total", [(64, 16, 1500), (64, 16, 8500), (64, 32, 8500), (64, 64, 2000), (128, 16, 8500),
                                        (128, 32, 1100), (128, 128, 1300), (128, 256, 1500)])
def test_append_large_batches(cuda_device, d, bs, total):
    """Whole blocks, parts of blocks and single tokens in a batch that is taken
    in larger spans, with padding between them; values over many magnitudes."""
    rng = np.random.default_rng(total + d + bs)
    runs, left = [], total
    while left > 0:
        n = min(left, int(rng.choice([1, 2, bs // 2, bs - 1, bs, bs, bs])))
        runs.append((int(rng.integers(0, bs - n + 1)), n))
        left -= n
    nb = len(runs) + 1
    slots = np.concatenate([blk * bs + r + np.arange(n) if i % 11 else np.full(n, -1)
                            for i, (blk, (r, n)) in enumerate(zip(rng.permutation(nb), runs))])
    kb, vb = (rng.integers(0, 127, (nb, 1, bs, d)).astype(np.uint8) for _ in range(2))
    ks, vs = (2.0 ** rng.integers(-12, 3, (nb, 1)) for _ in range(2))
    kt, vt = (bf16(rng.normal(size=(total, 1, d)) * 2.0 ** rng.integers(-9, 9, (total, 1, 1)), cuda_device)
              for _ in range(2))
    got = run_append(kt, vt, kb, vb, ks, vs, slots, cuda_device)
    for x, b0, s0, gb, gs in ((kt, kb, ks, got[0], got[2]), (vt, vb, vs, got[1], got[3])):
        wb, ws = P.append(x.double().cpu().numpy(), b0, s0, slots)
        np.testing.assert_array_equal(gs, ws.astype(np.float32))
        same_bytes(gb, wb)


def test_append_special_values(cuda_device):
    """Zeros, subnormal and huge values, infinities and NaN; scales so far that
    are no powers of two, zero, or not finite; padding and slots out of range."""
    d, bs, H, nb = 64, 16, 1, 8
    x = np.zeros((8, H, d))
    x[1] = 1e-40
    x[2] = 3.3e38
    x[3, 0, :4] = [np.inf, -np.inf, np.nan, 2.0]
    x[4] = np.inf
    x[5] = np.linspace(-1, 1, d)
    x[6] = 5.0
    x[7] = 1.0
    slots = [0, bs, 2 * bs, 3 * bs, 4 * bs + 1, 5 * bs + 2, -1, nb * bs]
    kb = np.random.default_rng(0).integers(0, 127, (nb, H, bs, d)).astype(np.uint8)
    ks = np.array([1, 1, 1, 1, 0.3, 0.003, 1, 1])[:, None]
    kt = bf16(x, cuda_device)
    got = run_append(kt, kt, kb, kb, ks, ks, slots, cuda_device)
    wb, ws = P.append(kt.double().cpu().numpy(), kb, ks, slots)
    np.testing.assert_array_equal(got[2], ws.astype(np.float32))
    same_bytes(got[0], wb)
    same_bytes(got[1], wb)
    assert got[2][0, 0] == 2.0 ** -126 and got[0][3, 0, 0, :2].tolist() == [126, 254]
    # a scale so far that is zero, infinite or NaN does not reach the new one
    for bad in (0.0, np.inf, np.nan, -1.0):
        got = run_append(kt[7:], kt[7:], kb, kb, np.full((nb, H), bad), np.full((nb, H), bad), [2 * bs + 5],
                         cuda_device)
        assert got[2][2, 0] == 2.0 ** -8
        assert (P.e4m3_decode(got[0][2, 0, 5]) == 256.0).all()
        np.testing.assert_array_equal(got[0][2, 0, 6:], kb[2, 0, 6:])


def test_append_nothing(cuda_device):
    c = fa.paged_cache(2, 1, 16, 64, 1, 2, cuda_device)
    e = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=cuda_device)
    fa.cache_append(e, e, c.k, c.v, c.k_scale, c.v_scale, torch.empty(0, dtype=torch.int32, device=cuda_device))
    assert fa.last_launch_count() == 0


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------

def make_cache(lens, bs, Hkv, d, seed, spread=1.0, scale_pow2=False):
    """Blocks in an arbitrary order, junk (NaN among it) in every row that
    holds no token and in every block that no table names."""
    rng = np.random.default_rng(seed)
    used = [-(-x // bs) for x in lens]
    nb = max(1, sum(used)) + 2
    mb = max(1, max(used))
    perm = rng.permutation(nb)
    table = np.full((len(lens), mb), -1, np.int32)
    kb, vb = (rng.integers(0, 256, (nb, Hkv, bs, d)).astype(np.uint8) for _ in range(2))
    at = 0
    for b, x in enumerate(lens):
        table[b, :used[b]] = perm[at:at + used[b]]
        at += used[b]
        for j in range(used[b]):
            r = min(bs, x - j * bs)
            for a in (kb, vb):
                a[table[b, j], :, :r] = P.e4m3_encode(rng.normal(size=(Hkv, r, d)) * 60)
    if scale_pow2:
        ks, vs = (2.0 ** rng.integers(-7, -4, (nb, Hkv)) for _ in range(2))
    else:
        ks, vs = (rng.uniform(0.3, 1.7, (nb, Hkv)) / 60 for _ in range(2))
    ks = (ks * spread).astype(np.float32)
    return kb, vb, ks, vs.astype(np.float32), table


def run_attend(q, c, cu, lens, max_new, causal, dev, scale, junk=7.0):
    kb, vb, ks, vs, table = c
    total, Hq, d = q.shape
    t = [torch.tensor(x, device=dev).view(torch.float8_e4m3fn) for x in (kb, vb)]
    s = [torch.tensor(x, device=dev) for x in (ks, vs)]
    o = torch.full_like(q, junk)
    lse = torch.full((Hq, total), junk, device=dev)
    ws = fa.workspace(fa.fwd_paged_workspace_size(len(lens), Hq, kb.shape[1], total, max_new, d), dev)
    fa.forward_paged(q, *t, *s, dev_i32(cu, dev), dev_i32(lens, dev), dev_i32(table, dev), max_new, scale=scale,
                     causal=causal, out=o, lse=lse, ws=ws)
    assert fa.get_status(ws) == fb.FA_OK
    return o.double().cpu().numpy(), lse.double().cpu().numpy()


def check(o, lse, ref, cu, G, rows, visible, d):
    """Bounds. Scores: d products and sums in fp32 (d 2^-24 of sum |q k|), the
    two scale factors and the exponent's argument (4 roundings of 2^-24), Q's
    f16 parts (2^-25 of the row's largest): together below (d + 16) 2^-24 X.
    Requests of more than 32 rows (24 at d = 128; new tokens x heads of a group; beside one of
    those, of more rows than a token has) take Q as two E4M3 parts: 2^-17 of the row's largest, hence 2^-17 Y more. Weights: f16 (2^-11), exp2 (2^-22) and twice the score error; weights below
    2^-31 of the largest vanish. O: that on A = sum P |v|, fp32 sums (2^-20 A),
    and bf16 (2^-8 |O|)."""
    O, L, A, X, Y = ref
    n, most = np.repeat(np.diff(cu), np.diff(cu))[rows], int(np.diff(cu).max()) * G
    cap = 32 if d == 64 else 24
    split = 8 * -(-(most if most <= cap else min(G, cap)) // 8)   # rows up to which Q is f16
    ds = (d + 16) * 2.0 ** -24 * X[:, rows] + np.where(n * G > split, 2.0 ** -17, 0.0) * Y[:, rows]
    L, lse = L[:, rows], lse[:, rows]
    empty = np.isneginf(L)
    assert np.array_equal(empty, np.isneginf(lse))
    with np.errstate(invalid="ignore"):
        el = np.where(empty, 0.0, np.abs(lse - L))
    tl = ds + 2.0 ** -18 + 2.0 ** -21 * np.abs(np.where(empty, 0.0, L))
    assert (el <= tl).all(), (el.max(), tl[el > tl].min())
    O, o, A = O[rows], o[rows], A[rows]
    w = (2.0 ** -11 + 2.0 ** -20 + 2 * ds + visible * 2.0 ** -31).T[..., None]
    eo, to = np.abs(o - O), 2.0 ** -8 * np.abs(O) + w * A * 1.01 + 1e-30
    assert (eo <= to).all(), ((eo / to).max(), np.argwhere(eo > to)[:5])
    assert (o[empty.T] == 0).all()


LENS = {
    "one": [(0, 1)],
    "short": [(999, 1)],
    "ragged": [(0, 1), (15, 1), (16, 1), (31, 1), (32, 1), (63, 1), (64, 1), (511, 1), (1500, 1), (2, 1)],
    "empty": [(40, 0), (12, 1), (0, 0), (77, 1)],
    "draft": [(100, 3), (0, 4), (31, 2), (255, 5), (64, 1)],
    "prompt": [(0, 130), (0, 7), (257, 65)],
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 256])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 4), (1, 7), (2, 8), (1, 12), (3, 1)])
@pytest.mark.parametrize("which", list(LENS))
def test_attend_within_bounds(cuda_device, d, bs, Hkv, G, which):
    if which == "prompt" and (bs, G) not in ((16, 1), (64, 4), (256, 7), (32, 12)):
        pytest.skip("long rows at some head layouts only")
    pairs = LENS[which]
    lens = [c + n for c, n in pairs]
    cu = np.concatenate([[0], np.cumsum([n for _, n in pairs])])
    total, pad = int(cu[-1]), 2
    rng = np.random.default_rng(d + bs + G)
    q = bf16(rng.normal(size=(total + pad, Hkv * G, d)), cuda_device)
    c = make_cache(lens, bs, Hkv, d, seed=bs + G)
    scale = 1 / math.sqrt(d)
    for causal in (True, False):
        o, lse = run_attend(q, c, cu, lens, max(n for _, n in pairs), causal, cuda_device, scale)
        ref = P.attend(q.double().cpu().numpy(), *c[:4], cu, lens, c[4], scale, causal)
        check(o, lse, ref, cu, G, slice(0, total), max(lens), d)
        assert (o[total:] == 7).all() and (lse[:, total:] == 7).all()   # rows behind the last request


@pytest.mark.parametrize("d", [64, 128])
def test_attend_peaked_and_flat_rows(cuda_device, d):
    """Scores from hundreds of binary orders down to none at all: the
    reference maximum moves, most weights vanish, or all are alike."""
    lens, cu = [1500, 700], [0, 2, 4]
    rng = np.random.default_rng(1)
    c = make_cache(lens, 64, 2, d, seed=2, spread=30.0)
    q = rng.normal(size=(4, 4, d)) * np.array([1e-3, 0, 1.0, 8.0])[:, None, None]
    q[1] = 0
    q = bf16(q, cuda_device)
    o, lse = run_attend(q, c, cu, lens, 2, True, cuda_device, 0.1)
    ref = P.attend(q.double().cpu().numpy(), *c[:4], cu, lens, c[4], 0.1)
    check(o, lse, ref, cu, 2, slice(0, 4), 1500, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,G", [(2, 8), (17, 1), (3, 8), (1, 24), (1, 25), (5, 5), (4, 8), (1, 32), (3, 11), (1, 33)])
def test_attend_rows_at_the_borders(cuda_device, d, n, G):
    """Requests of just as many rows as a tile of either kernel takes, one more,
    and fewer beside them."""
    lens, cu = [n + 40, n + 900, 31, n, 500], np.concatenate([[0], np.cumsum([n, n, 1, n, 0])])
    rng = np.random.default_rng(d + n + G)
    c = make_cache(lens, 32, 2, d, seed=n + G)
    q = bf16(rng.normal(size=(int(cu[-1]), 2 * G, d)), cuda_device)
    o, lse = run_attend(q, c, cu, lens, n, True, cuda_device, 0.1)
    ref = P.attend(q.double().cpu().numpy(), *c[:4], cu, lens, c[4], 0.1)
    check(o, lse, ref, cu, G, slice(0, int(cu[-1])), max(lens), d)


def test_attend_long_cache_of_one_request(cuda_device):
    """One request over every CTA, cut into many pieces."""
    lens, cu, d = [40000], [0, 1], 128
    rng = np.random.default_rng(1)
    c = make_cache(lens, 64, 1, d, seed=2)
    q = bf16(rng.normal(size=(1, 8, d)), cuda_device)
    o, lse = run_attend(q, c, cu, lens, 1, True, cuda_device, 0.09)
    ref = P.attend(q.double().cpu().numpy(), *c[:4], cu, lens, c[4], 0.09)
    check(o, lse, ref, cu, 8, slice(0, 1), 40000, d)


def test_attend_many_requests(cuda_device):
    rng = np.random.default_rng(7)
    n = rng.integers(0, 3, 700)
    lens = (n + rng.integers(0, 90, 700)).tolist()
    cu = np.concatenate([[0], np.cumsum(n)])
    c = make_cache(lens, 16, 2, 64, seed=3)
    q = bf16(rng.normal(size=(int(cu[-1]), 4, 64)), cuda_device)
    o, lse = run_attend(q, c, cu, lens, 2, True, cuda_device, 0.125)
    ref = P.attend(q.double().cpu().numpy(), *c[:4], cu, lens, c[4], 0.125)
    check(o, lse, ref, cu, 2, slice(0, int(cu[-1])), 100, 64)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 128, 256])
@pytest.mark.parametrize("Hkv,G,pairs", [
    (1, 1, [(0, 33)]), (2, 1, [(0, 300), (7, 1), (1000, 129)]), (1, 8, [(5, 5), (130, 32), (600, 1), (0, 33)]),
    (1, 5, [(100, 52), (0, 0), (127, 26), (128, 26)]), (1, 40, [(300, 1), (77, 2)])])
def test_attend_many_rows(cuda_device, d, bs, Hkv, G, pairs):
    """Prompts and pieces of prompts beside requests of a few rows."""
    lens = [c + n for c, n in pairs]
    cu = np.concatenate([[0], np.cumsum([n for _, n in pairs])])
    total = int(cu[-1])
    rng = np.random.default_rng(d + bs + G)
    q = bf16(rng.normal(size=(total + 3, Hkv * G, d)), cuda_device)
    c = make_cache(lens, bs, Hkv, d, seed=bs + G)
    scale = 1 / math.sqrt(d)
    for causal in (True, False):
        o, lse = run_attend(q, c, cu, lens, max(n for _, n in pairs), causal, cuda_device, scale)
        ref = P.attend(q.double().cpu().numpy(), *c[:4], cu, lens, c[4], scale, causal)
        check(o, lse, ref, cu, G, slice(0, total), max(lens), d)
        assert (o[total:] == 7).all() and (lse[:, total:] == 7).all()


@pytest.mark.parametrize("d,Hkv,G,pairs", [
    (64, 16, 1, [(0, 1871), (0, 685), (0, 448), (0, 1255), (0, 314), (0, 1967), (0, 1054), (0, 1142)]),
    (128, 8, 4, [(3000, 700), (0, 900), (515, 333)])])
def test_attend_prompts_again_and_again(cuda_device, d, Hkv, G, pairs):
    """Many row tiles in every CTA, twenty times: the same bits each time, and
    within the sum of the bounds (here 2^-7 of a row's largest value, bf16's
    2^-8 and as much for P and the scores) of a float64 computation."""
    lens = [c + n for c, n in pairs]
    cu = np.concatenate([[0], np.cumsum([n for _, n in pairs])])
    total, bs, scale = int(cu[-1]), 64, 1 / math.sqrt(d)
    gen = torch.Generator(device=cuda_device).manual_seed(3)
    used = [-(-x // bs) for x in lens]
    perm = torch.randperm(sum(used), generator=gen, device=cuda_device).to(torch.int32)
    table = torch.full((len(lens), max(used)), -1, dtype=torch.int32, device=cuda_device)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
    kc, vc = ((torch.randn((at, Hkv, bs, d), generator=gen, device=cuda_device) * 60).to(torch.float8_e4m3fn)
              for _ in range(2))
    ks, vs = (torch.ldexp(torch.ones((at, Hkv), device=cuda_device),
                          torch.randint(-7, -4, (at, Hkv), generator=gen, device=cuda_device)) for _ in range(2))
    q = torch.randn((total, Hkv * G, d), generator=gen, device=cuda_device).to(torch.bfloat16)
    args = (q, kc, vc, ks, vs, dev_i32(cu, cuda_device), dev_i32(lens, cuda_device), table,
            max(n for _, n in pairs))
    o, lse = fa.forward_paged(*args, scale=scale)
    for _ in range(20):
        again = fa.forward_paged(*args, scale=scale)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    for b, (c, n) in enumerate(pairs):
        t = table[b, :used[b]].long()
        seen = torch.arange(lens[b], device=cuda_device) <= c + torch.arange(n, device=cuda_device)[:, None]
        for h in range(Hkv):
            k, v = ((x[t, h].double() * s[t, h].double()[:, None, None]).reshape(-1, d)[:lens[b]]
                    for x, s in ((kc, ks), (vc, vs)))
            for g in range(h * G, (h + 1) * G):
                x = torch.where(seen, (q[cu[b]:cu[b + 1], g].double() @ k.T) * scale, -math.inf)
                want = torch.softmax(x, -1) @ v
                err = (o[cu[b]:cu[b + 1], g].double() - want).abs()
                assert (err <= 2.0 ** -7 * v.abs().max(0).values).all(), (b, g)


def test_attend_many_rows_over_a_long_cache(cuda_device):
    """One piece of a prompt, its keys split over every CTA."""
    lens, cu, d = [20000], [0, 40], 128
    rng = np.random.default_rng(1)
    c = make_cache(lens, 64, 1, d, seed=2)
    q = bf16(rng.normal(size=(40, 2, d)), cuda_device)
    o, lse = run_attend(q, c, cu, lens, 40, True, cuda_device, 0.09)
    ref = P.attend(q.double().cpu().numpy(), *c[:4], cu, lens, c[4], 0.09)
    check(o, lse, ref, cu, 2, slice(0, 40), 20000, d)
    again = run_attend(q, c, cu, lens, 40, True, cuda_device, 0.09)
    np.testing.assert_array_equal(o, again[0])
    np.testing.assert_array_equal(lse, again[1])


@pytest.mark.parametrize("n", [1, 40])
def test_attend_block_scales_far_apart(cuda_device, n):
    """Blocks of zeros (scale 2^-126 or 0), values 2^20 apart, key scales from
    none to large, and weights that lie on the small values."""
    lens, cu, d, bs = [333], [0, n], 64, 16
    rng = np.random.default_rng(6)
    kb, vb, ks, vs, table = make_cache(lens, bs, 1, d, seed=2)
    blocks = table[0]
    vs[blocks, 0] = (2.0 ** rng.integers(-12, 9, len(blocks))).astype(np.float32)
    for i, z in ((0, 2.0 ** -126), (3, 0.0), (20, 2.0 ** -126)):
        vs[blocks[i], 0] = z
        vb[blocks[i]] = 0
    ks[blocks, 0] = (rng.uniform(0, 0.2, len(blocks))).astype(np.float32)
    ks[blocks[5], 0] = 0.0
    ks[blocks[0], 0] = 2.0 ** -126
    kb[blocks[0]] = 0
    q = bf16(rng.normal(size=(n, 2, d)), cuda_device)
    c = (kb, vb, ks, vs, table)
    o, lse = run_attend(q, c, cu, lens, n, True, cuda_device, 0.1)
    ref = P.attend(q.double().cpu().numpy(), *c[:4], cu, lens, table, 0.1)
    check(o, lse, ref, cu, 2, slice(0, n), 333, d)
    vb[blocks] = 0                                   # nothing but zeros
    vs[blocks, 0] = 2.0 ** -126
    o, lse2 = run_attend(q, c, cu, lens, n, True, cuda_device, 0.1)
    assert (o == 0).all()
    np.testing.assert_allclose(lse2, lse, rtol=1e-5)


def test_attend_refused_request_and_rows_that_see_nothing(cuda_device):
    """A request whose tokens are not in the cache: more rows than tokens."""
    lens, cu = [3, 0, 20], [0, 5, 7, 8]
    rng = np.random.default_rng(9)
    c = make_cache(lens, 16, 1, 64, seed=3)
    q = bf16(rng.normal(size=(8, 2, 64)), cuda_device)
    for causal in (True, False):
        o, lse = run_attend(q, c, cu, lens, 5, causal, cuda_device, 0.125)
        ref = P.attend(q.double().cpu().numpy(), *c[:4], cu, lens, c[4], 0.125, causal)
        check(o, lse, ref, cu, 2, slice(0, 8), 20, 64)


@pytest.mark.parametrize("d,G,n", [(128, 2, 4), (64, 4, 8), (128, 8, 70), (64, 1, 130)])
@pytest.mark.parametrize("old", [0, 200])
def test_attend_nan_reaches_only_the_rows_that_see_it(cuda_device, d, G, n, old):
    """NaN in new tokens' values and keys: rows before them stay finite."""
    lens, cu = [old + n], [0, n]
    rng = np.random.default_rng(4)
    kb, vb, ks, vs, table = make_cache(lens, 32, 1, d, seed=8)

    def put(a, pos, col):
        a[table[0, pos // 32], 0, pos % 32, col] = 0x7F if pos % 2 else 0xFF

    first_v, first_k = old + n // 2, old + n - 1
    put(vb, first_v, 5)
    put(vb, first_v + 1, 5)
    put(vb, first_v + 1, d - 1)
    put(kb, first_k, 3)
    q = bf16(rng.normal(size=(n, G, d)), cuda_device)
    c = (kb, vb, ks, vs, table)
    o, lse = run_attend(q, c, cu, lens, n, True, cuda_device, 0.125)
    for i in range(n):
        pos = old + i
        nan = np.zeros(d, bool)
        if pos >= first_v:
            nan[5] = True
        if pos >= first_v + 1:
            nan[d - 1] = True
        if pos >= first_k:
            nan[:] = True
        assert (np.isnan(o[i]) == nan).all(), i
        assert (np.isnan(lse[:, i]) == (pos >= first_k)).all()
    rows = slice(0, n // 2)                    # before the first NaN: exact as ever
    ref = P.attend(q.double().cpu().numpy()[rows], *c[:4], [0, n // 2], [old + n // 2], table, 0.125)
    check(o, lse, ref, cu, G, rows, old + n, d)


def test_attend_infinite_and_nan_queries_stay_in_their_rows(cuda_device):
    lens, cu = [70], [0, 1]
    c = make_cache(lens, 32, 1, 128, seed=8)
    q = np.random.default_rng(0).normal(size=(1, 4, 128))
    q[0, 1, 7], q[0, 3, 9] = np.inf, np.nan
    o, lse = run_attend(bf16(q, cuda_device), c, cu, lens, 1, True, cuda_device, 0.1)
    assert np.isnan(o[0, [1, 3]]).all() and np.isfinite(o[0, [0, 2]]).all() and np.isfinite(lse[[0, 2]]).all()


def test_attend_reports_bad_tables(cuda_device):
    lens, cu, d = [100, 60], [0, 1, 2], 64
    kb, vb, ks, vs, table = make_cache(lens, 16, 1, d, seed=8)
    q = bf16(np.random.default_rng(0).normal(size=(2, 2, d)), cuda_device)
    good = run_attend(q, (kb, vb, ks, vs, table), cu, lens, 1, True, cuda_device, 0.1)

    def status(table=table, cu=cu, lens=lens, max_new=1):
        t = [torch.tensor(x, device=cuda_device).view(torch.float8_e4m3fn) for x in (kb, vb)]
        s = [torch.tensor(x, device=cuda_device) for x in (ks, vs)]
        ws = fa.workspace(fa.fwd_paged_workspace_size(2, 2, 1, 2, max_new, d), cuda_device)
        o, _ = fa.forward_paged(q, *t, *s, dev_i32(cu, cuda_device), dev_i32(lens, cuda_device),
                                dev_i32(table, cuda_device), max_new, scale=0.1, ws=ws)
        return fa.get_status(ws), o.double().cpu().numpy()

    assert status()[0] == fb.FA_OK
    for v in (-1, kb.shape[0], 1 << 30, -(1 << 31)):
        bad = table.copy()
        bad[0, 3] = v
        st, o = status(table=bad)
        assert st == fb.FA_ERR_INVALID_ARG
        np.testing.assert_array_equal(o[1], good[0][1])        # the other request is not touched
    assert status(lens=[100, 1 << 30])[0] == fb.FA_ERR_INVALID_ARG
    assert status(lens=[-3, 60])[0] == fb.FA_ERR_INVALID_ARG
    assert status(cu=[0, 2, 1])[0] == fb.FA_ERR_INVALID_ARG
    assert status(cu=[0, 2, 2])[0] == fb.FA_ERR_INVALID_ARG    # two tokens, max_new = 1
    assert status(cu=[-4, 1, 9])[0] == fb.FA_ERR_INVALID_ARG


def test_attend_is_deterministic_and_ignores_what_lies_behind(cuda_device):
    pairs = [(1000, 2), (40, 1), (3000, 2)]
    lens = [c + n for c, n in pairs]
    cu = [0, 2, 3, 5]
    rng = np.random.default_rng(2)
    q = bf16(rng.normal(size=(5, 8, 128)), cuda_device)
    c = make_cache(lens, 64, 2, 128, seed=1)
    a = run_attend(q, c, cu, lens, 2, True, cuda_device, 0.1)
    b = run_attend(q, c, cu, lens, 2, True, cuda_device, 0.1)
    np.testing.assert_array_equal(a[0], b[0])
    np.testing.assert_array_equal(a[1], b[1])
    kb, vb = c[0].copy(), c[1].copy()
    for r, x in enumerate(lens):
        if x % 64:
            for z in (kb, vb):
                z[c[4][r, x // 64], :, x % 64:] = 0x7F
    d = run_attend(q, (kb, vb, *c[2:]), cu, lens, 2, True, cuda_device, 0.1)
    np.testing.assert_array_equal(a[0], d[0])
    np.testing.assert_array_equal(a[1], d[1])


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------

def serve_state(dev, bs=16, Hkv=2, d=64, B=5, nb=60, mb=20):
    return fa.paged_cache(nb, Hkv, bs, d, B, mb, dev)


def oracle_step(s, new, k, v, q, bs, total, scale):
    r = P.plan(new, s["cache_len"], s["block_table"], s["free_blocks"], s["free_state"], bs, total)
    s.update({x: r[x] for x in ("cache_len", "block_table", "free_blocks", "free_state")})
    s["kb"], s["ks"] = P.append(k, s["kb"], s["ks"], r["slots"])
    s["vb"], s["vs"] = P.append(v, s["vb"], s["vs"], r["slots"])
    return r, P.attend(q, s["kb"], s["vb"], s["ks"], s["vs"], r["cu_seqlens"], s["cache_len"], s["block_table"], scale)


def oracle_state(nb, Hkv, bs, d, B, mb):
    return dict(cache_len=np.zeros(B, np.int32), block_table=np.full((B, mb), -1, np.int32),
                free_blocks=np.arange(nb, dtype=np.int32), free_state=np.array([0, nb], np.int32),
                kb=np.zeros((nb, Hkv, bs, d), np.uint8), vb=np.zeros((nb, Hkv, bs, d), np.uint8),
                ks=np.zeros((nb, Hkv)), vs=np.zeros((nb, Hkv)))


def test_serving_steps(cuda_device):
    """Prompts, decoding, drafts, a release and a request that takes its
    place, a request that finds no blocks: plan, append and attend in turn."""
    bs, Hkv, G, d, B, nb, mb = 16, 2, 3, 64, 5, 24, 20
    c = serve_state(cuda_device, bs, Hkv, d, B, nb, mb)
    s = oracle_state(nb, Hkv, bs, d, B, mb)
    rng = np.random.default_rng(11)
    steps = [[40, 7, 0, 16, 1], [1, 1, 33, 1, 1], [1, 3, 1, 2, 1], [-1, 1, 1, 1, 1], [50, 1, 0, 1, 1],
             [1, 1, 1, 90, 1], [1, -1, 1, 90, 1], [1, 20, 1, 90, 1], [1, 1, 1, 1, 1]]
    refused = 0
    for new in steps:
        total = sum(max(x, 0) for x in new) + 1                     # one padding row
        grow = 2.0 ** rng.integers(-2, 4, (total, 1, 1))
        k, v = (bf16(rng.normal(size=(total, Hkv, d)) * grow, cuda_device) for _ in range(2))
        q = bf16(rng.normal(size=(total, Hkv * G, d)), cuda_device)
        ws = fa.workspace(256, cuda_device)
        cu, slots = fa.cache_plan(dev_i32(new, cuda_device), c.cache_len, c.block_table, c.free_blocks, c.free_state,
                                  bs, total=total, ws=ws)
        st = fa.get_status(ws)
        fa.cache_append(k, v, c.k, c.v, c.k_scale, c.v_scale, slots)
        o, lse = fa.forward_paged(q, c.k, c.v, c.k_scale, c.v_scale, cu, c.cache_len, c.block_table,
                                  max(max(new), 0), scale=0.125)
        r, ref = oracle_step(s, new, *(x.double().cpu().numpy() for x in (k, v, q)), bs, total, 0.125)
        for name, t in (("slots", slots), ("cu_seqlens", cu), ("cache_len", c.cache_len),
                        ("block_table", c.block_table), ("free_blocks", c.free_blocks), ("free_state", c.free_state)):
            np.testing.assert_array_equal(t.cpu().numpy(), r[name], err_msg=name)
        assert st == (fb.FA_ERR_NO_BLOCKS if r["refused"] else fb.FA_OK)
        refused += len(r["refused"])
        same_bytes(c.k.view(torch.uint8).cpu().numpy(), s["kb"])
        same_bytes(c.v.view(torch.uint8).cpu().numpy(), s["vb"])
        np.testing.assert_array_equal(c.k_scale.cpu().numpy(), s["ks"].astype(np.float32))
        check(o.double().cpu().numpy(), lse.double().cpu().numpy(), ref, r["cu_seqlens"], G,
              slice(0, total - 1), 400, d)
    assert refused > 0


def test_serving_step_in_a_graph(cuda_device):
    """One captured decoding step replayed: lengths, tables and the cache move
    on in place; the result equals eager calls on a twin."""
    bs, Hkv, G, d, B = 32, 2, 4, 128, 6
    gen = torch.Generator(device=cuda_device).manual_seed(0)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device=cuda_device).to(torch.bfloat16)

    new = torch.ones(B, dtype=torch.int32, device=cuda_device)
    q, k, v = rand(B, Hkv * G, d), rand(B, Hkv, d), rand(B, Hkv, d)
    caches = [fa.paged_cache(64, Hkv, bs, d, B, 16, cuda_device) for _ in range(2)]
    prompt = torch.tensor([5, 31, 32, 33, 100, 64], dtype=torch.int32, device=cuda_device)
    n0 = int(prompt.sum())
    pk, pv, pq = rand(n0, Hkv, d), rand(n0, Hkv, d), rand(n0, Hkv * G, d)

    def step(c, new, total, q, k, v, max_new, bufs):
        cu, slots = fa.cache_plan(new, c.cache_len, c.block_table, c.free_blocks, c.free_state, bs, total=total,
                                  cu_seqlens=bufs["cu"], slots=bufs.get("slots"), ws=bufs["wp"])
        fa.cache_append(k, v, c.k, c.v, c.k_scale, c.v_scale, slots)
        return fa.forward_paged(q, c.k, c.v, c.k_scale, c.v_scale, cu, c.cache_len, c.block_table, max_new,
                                out=bufs.get("o"), lse=bufs.get("lse"), ws=bufs.get("ws"))

    i32 = dict(dtype=torch.int32, device=cuda_device)
    bufs = [dict(cu=torch.empty(B + 1, **i32), wp=fa.workspace(256, cuda_device)) for _ in range(2)]
    first = [step(c, prompt, n0, pq, pk, pv, 100, b) for c, b in zip(caches, bufs)]
    assert torch.equal(first[0][0], first[1][0])
    for b in bufs:
        b.update(slots=torch.empty(B, **i32), o=torch.empty_like(q), lse=torch.empty((Hkv * G, B), device=cuda_device),
                 ws=fa.workspace(fa.fwd_paged_workspace_size(B, Hkv * G, Hkv, B, 1, d), cuda_device))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c, b in zip(caches, bufs):
            step(c, new, B, q, k, v, 1, b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0], new, B, q, k, v, 1, bufs[0])
    for i in range(40):
        for t in (q, k, v):
            t.copy_(rand(*t.shape))
        graph.replay()
        step(caches[1], new, B, q, k, v, 1, bufs[1])
        assert torch.equal(bufs[0]["o"], bufs[1]["o"]) and torch.equal(bufs[0]["lse"], bufs[1]["lse"]), i
    for x, y in zip(caches[0], caches[1]):
        x, y = (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in (x, y))
        assert torch.equal(x, y)
    assert caches[0].cache_len.tolist() == [x + 41 for x in prompt.tolist()]
    assert fa.get_status(bufs[0]["wp"]) == fb.FA_OK and fa.get_status(bufs[0]["ws"]) == fb.FA_OK


def test_two_streams_at_once(cuda_device):
    """Two calls in flight with a workspace each."""
    pairs = [(3000, 1)] * 8
    lens, cu = [c + n for c, n in pairs], list(range(9))
    rng = np.random.default_rng(2)
    c = make_cache(lens, 64, 2, 128, seed=1)
    t = [torch.tensor(x, device=cuda_device).view(torch.float8_e4m3fn) for x in c[:2]]
    s = [torch.tensor(x, device=cuda_device) for x in c[2:4]]
    args = (*t, *s, dev_i32(cu, cuda_device), dev_i32(lens, cuda_device), dev_i32(c[4], cuda_device), 1)
    qs = [bf16(rng.normal(size=(8, 16, 128)), cuda_device) for _ in range(2)]
    want = [fa.forward_paged(q, *args) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(5):
        for q, st in zip(qs, streams):
            with torch.cuda.stream(st):
                outs.append(fa.forward_paged(q, *args))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(outs):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])
