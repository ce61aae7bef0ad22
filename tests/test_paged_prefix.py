"""GPU checks of attention over the paged cache with shared prefixes against
the fp64 oracle."""

import math

import numpy as np
import pytest
import torch

import io_aware_exact_tiled_gb300 as fa
from io_aware_exact_tiled_gb300 import binding as fb
from oracle import paged_prefix as PP

from test_paged import bf16, dev_i32, make_cache

pytestmark = pytest.mark.gpu


class Batch:
    """Requests (cached, new tokens) in groups [(first request, prefix length)];
    requests in front of the first group have no prefix, nor those from `stop` on."""

    def __init__(self, pairs, groups, bs, Hkv, G, d, device, seed=0, stop=None, pad=2, spread=1.0):
        self.lens, self.new = [c + n for c, n in pairs], [n for _, n in pairs]
        self.cu = np.concatenate([[0], np.cumsum(self.new)])
        self.pcu = [g[0] for g in groups] + [len(pairs) if stop is None else stop]
        self.plen = [g[1] for g in groups]
        self.Hkv, self.G, self.d, self.dev = Hkv, G, d, device
        *self.c, table = make_cache(self.lens + self.plen, bs, Hkv, d, seed, spread=spread)
        self.table, self.ptable = table[: len(pairs)], table[len(pairs):]
        self.total = int(self.cu[-1])
        rng = np.random.default_rng(seed + d)
        self.q = bf16(rng.normal(size=(self.total + pad, Hkv * G, d)), device)
        self.scale = 1 / math.sqrt(d)

    def tensors(self):
        kb, vb, ks, vs = self.c
        t = [torch.tensor(x, device=self.dev).view(torch.float8_e4m3fn) for x in (kb, vb)]
        t += [torch.tensor(x, device=self.dev) for x in (ks, vs)]
        return t + [dev_i32(x, self.dev) for x in (self.cu, self.lens, self.table, self.pcu, self.plen, self.ptable)]

    def run(self, causal=True, ws=None, args=None, status=fb.FA_OK):
        n, Hq = self.q.shape[0], self.Hkv * self.G
        o = torch.full_like(self.q, 7.0)
        lse = torch.full((Hq, n), 7.0, device=self.dev)
        if ws is None:
            size = fa.fwd_paged_prefix_workspace_size(len(self.lens), len(self.plen), Hq, self.Hkv, n, max(self.new),
                                                      self.d)
            ws = fa.workspace(size, self.dev).fill_(255)
        fa.forward_paged_prefix(self.q, *(args or self.tensors()), max(self.new), scale=self.scale, causal=causal, out=o,
                                lse=lse, ws=ws)
        assert fa.get_status(ws) == status
        return o, lse

    def check(self, causal=True, got=None):
        """Bounds. Scores, weights and sums of a part are forward_paged's
        (tests of its own state them), Q taken as two E4M3 parts where that is
        the larger error: (d + 16) 2^-24 X + 2^-17 Y. Joining two parts: the
        difference of maxima and of two logarithms (2^-22 each), exp2, a
        division and three products: below 2^-19."""
        o, lse = (x.double().cpu().numpy() for x in (got or self.run(causal)))
        assert (o[self.total:] == 7).all() and (lse[:, self.total:] == 7).all()
        o, lse = o[: self.total], lse[:, : self.total]
        O, L, A, X, Y = PP.attend(self.q.double().cpu().numpy()[: self.total], *self.c, self.cu, self.lens, self.table,
                                  self.pcu, self.plen, self.ptable, self.scale, causal)
        ds = (self.d + 16) * 2.0 ** -24 * X + 2.0 ** -17 * Y
        empty = np.isneginf(L)
        assert np.array_equal(empty, np.isneginf(lse))
        with np.errstate(invalid="ignore"):
            el = np.where(empty, 0.0, np.abs(lse - L))
        tl = ds + 2.0 ** -18 + 2.0 ** -21 * np.abs(np.where(empty, 0.0, L))
        assert (el <= tl).all(), (el / tl).max()
        seen = max(self.lens) + max(self.plen)
        w = (2.0 ** -11 + 2.0 ** -19 + 2 * ds + seen * 2.0 ** -31).T[..., None]
        eo, to = np.abs(o - O), 2.0 ** -8 * np.abs(O) + w * A * 1.01 + 1e-30
        assert (eo <= to).all(), ((eo / to).max(), np.argwhere(eo > to)[:5])
        assert (o[empty.T] == 0).all()


BATCHES = {
    # requests, groups
    "one": ([(0, 1)], [(0, 1)], None),
    "decode": ([(9, 1), (40, 1), (0, 1), (700, 1), (64, 1)], [(0, 333)], None),
    "groups": ([(3, 1), (1, 2), (77, 1), (0, 1), (32, 1), (5, 3), (200, 1)], [(0, 64), (2, 0), (3, 500), (5, 31)], None),
    # requests without a prefix in front and behind, a request without new tokens, an empty group
    "outside": ([(20, 1), (3, 1), (9, 0), (100, 2), (0, 1), (8, 1)], [(1, 100), (2, 40), (2, 7), (4, 33)], 5),
    # no own tokens cached: the prefix alone, or nothing at all
    "no own": ([(-1, 1), (5, 1), (-2, 2), (-1, 1)], [(0, 50), (3, 0)], None),
    "many rows": ([(i * 7 % 50, 1 + i % 4) for i in range(40)], [(0, 700), (25, 150)], None),
    "prompts": ([(0, 130), (10, 7), (0, 300), (257, 65)], [(0, 200), (2, 129)], None),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs,Hkv,G", [(16, 1, 1), (64, 2, 4), (128, 1, 8), (32, 3, 2), (256, 1, 12)])
@pytest.mark.parametrize("which", list(BATCHES))
def test_within_bounds(cuda_device, which, bs, Hkv, G, d):
    pairs, groups, stop = BATCHES[which]
    b = Batch(pairs, groups, bs, Hkv, G, d, cuda_device, seed=bs + G, stop=stop)
    for causal in (True, False):
        b.check(causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,G", [(1, 8), (2, 8), (3, 8), (4, 8), (5, 8), (16, 8), (32, 8), (33, 8), (3, 11)])
def test_rows_at_the_borders(cuda_device, B, G, d):
    """As many rows as the tiles take, one more, one less."""
    Batch([(i, 1) for i in range(B)], [(0, 900)], 32, 1, G, d, cuda_device, seed=B).check()
    Batch([(i, 1) for i in range(B + 2)], [(0, 0), (1, 900), (B + 1, 40)], 32, 1, G, d, cuda_device, seed=B).check()


@pytest.mark.parametrize("d,B", [(128, 2), (64, 12), (128, 40)])
def test_a_long_prefix(cuda_device, d, B):
    """One prefix over every CTA, cut into many pieces."""
    Batch([(i % 9, 1) for i in range(B)], [(0, 30000)], 64, 1, 4, d, cuda_device, seed=B).check()


def test_a_prefix_that_is_the_requests_own(cuda_device):
    """The blocks of a prefix and of a request may be the same ones."""
    b = Batch([(63, 1), (20, 1)], [(0, 64)], 16, 1, 4, 64, cuda_device)
    b.ptable = b.table[:1].copy()
    b.check()


@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_very_different_parts(cuda_device, d):
    """Either part may have all the weight."""
    for part in (0, 1):
        b = Batch([(40, 1), (60, 2)], [(0, 90)], 16, 2, 4, d, cuda_device, spread=4.0)
        at = b.ptable if part else b.table
        b.c[2][at[at >= 0]] *= 8.0
        b.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("more,new", [(0, 1), (9, 1), (30, 1), (70, 1), (2, 150)])
def test_nan_and_infinite_values(cuda_device, more, new, d):
    """A NaN of the prefix reaches all rows of its group and no other, one of a
    request's own tokens that request's; a query with an infinity has no finite
    row. With rows for every kernel and way of joining."""
    b = Batch([(40, 1), (60, 2), (9, 1)] + [(20, new)] * more, [(0, 90), (2, 50)], 16, 1, 4, d, cuda_device, pad=0)
    b.c[1][b.ptable[0, 5], 0, 9, 3] = 127              # token 89, the prefix's last
    b.c[1][b.table[2, 0], 0, 9, 7] = 127               # the third request's last
    b.q[3, 1, 0] = float("inf")
    o, lse = b.run()
    nan = o.isnan()
    assert nan[:3, :, 3].all() and nan[3, :, 7].all() and nan[3, 1].all()
    assert int(nan.sum()) == 12 + 3 + d
    assert lse[1, 3].isnan() and int(lse.isnan().sum()) == 1


@pytest.mark.parametrize("d", [64, 128])
def test_a_prefix_of_one_tile_behind_a_call_of_nans(cuda_device, d):
    """What another call left in tensor memory has no influence: a prefix of one
    key tile gives the second of a unit's two streams of keys nothing to do."""
    wild = Batch([(20, 1)] * 40, [(0, 30000)], 64, 4, 4, d, cuda_device, pad=0)
    wild.q.fill_(float("inf"))
    b = Batch([(9, 1)] * 20, [(0, 100)], 64, 8, 4, d, cuda_device)
    assert wild.run()[0].isnan().all()
    o, lse = b.run()
    b.check(got=(o, lse))


def test_no_prefix_is_forward_paged(cuda_device):
    """Groups without tokens: what forward_paged computes, whose work may be cut
    elsewhere, so that sums run in another order: both within the bounds."""
    b = Batch(BATCHES["groups"][0], [(0, 0), (3, 0)], 32, 2, 4, 128, cuda_device, pad=0)
    b.check()
    t = b.tensors()
    b.check(got=fa.forward_paged(b.q, *t[:7], max(b.new), scale=b.scale))


@pytest.mark.parametrize("which,d", [("many rows", 128), ("prompts", 64), ("groups", 64)])
def test_the_same_bits_each_time(cuda_device, which, d):
    pairs, groups, stop = BATCHES[which]
    b = Batch(pairs, [(g, 5 * n) for g, n in groups], 64, 4, 4, d, cuda_device, stop=stop)
    o, lse = b.run()
    b.check(got=(o, lse))
    for _ in range(5):
        p, pl = b.run()
        assert torch.equal(o, p) and torch.equal(lse, pl)


@pytest.mark.parametrize("more", [0, 40])
def test_offsets_and_lengths_out_of_range_are_reported(cuda_device, more):
    """In the split-key kernel's prefixes and in the row-tile kernel's."""
    bad = fb.FA_ERR_INVALID_ARG

    def batch():
        b = Batch([(40, 1), (60, 2), (9, 1)] + [(5, 1)] * more, [(0, 90), (2, 50)], 16, 1, 4, 64, cuda_device)
        return b, b.tensors()

    n = 3 + more
    for i, value in ((7, [0, n + 9, n]), (7, [0, 2, 1]), (7, [-1, 1, n]), (8, [1 << 20, 5]), (8, [-3, 5])):
        b, t = batch()
        t[i] = dev_i32(value, cuda_device)
        b.run(args=t, status=bad)
    for i, at in ((9, (0, 2)), (6, (1, 1))):          # table entries that are no block
        for value in (-1, 1 << 28):
            b, t = batch()
            t[i][at] = value
            b.run(args=t, status=bad)
    # behind the lengths anything may stand
    b, _ = batch()
    b.ptable[1, 4:] = 1 << 28
    b.check()


def test_a_serving_step_captured_and_replayed(cuda_device):
    """Plan, norm with append, and attention over a shared prefix in one graph,
    three steps of it, against the calls made one by one."""
    d, bs, Hkv, G, B, nb = 64, 16, 2, 4, 6, 64
    Hq = Hkv * G
    rng = np.random.default_rng(0)
    f = torch.tensor(1e4 ** (-np.arange(0, d, 2) / d), device=cuda_device)
    w = [bf16(1 + 0.2 * rng.normal(size=d), cuda_device) for _ in range(2)]
    pre_len, pre_blocks = 100, 7
    caches = []
    for _ in range(2):
        c = fa.paged_cache(nb, Hkv, bs, d, B, 8, cuda_device)
        c.free_state.copy_(dev_i32([pre_blocks, nb - pre_blocks], cuda_device))     # the prefix has the first blocks
        caches.append(c)
    cu1 = dev_i32([0, pre_len], cuda_device)
    pqkv = bf16(rng.normal(size=(pre_len, Hq + 2 * Hkv, d)), cuda_device)
    ptable = dev_i32([list(range(pre_blocks))], cuda_device)
    pcu, plen = dev_i32([0, B], cuda_device), dev_i32([pre_len], cuda_device)
    for c in caches:
        q, k, v = pqkv.split([Hq, Hkv, Hkv], 1)
        fa.qk_norm_rope_append(q, k, v, c.k, c.v, c.k_scale, c.v_scale, torch.arange(pre_len, device=cuda_device,
                               dtype=torch.int32), f, cu1, q_weight=w[0], k_weight=w[1])
    new = dev_i32([1] * B, cuda_device)
    qkv = bf16(np.zeros((B, Hq + 2 * Hkv, d)), cuda_device)
    steps = [bf16(rng.normal(size=qkv.shape), cuda_device) for _ in range(20)]
    ends = [torch.empty(B, dtype=torch.int32, device=cuda_device) for _ in range(2)]
    ws = [fa.workspace(fa.fwd_paged_prefix_workspace_size(B, 1, Hq, Hkv, B, 1, d), cuda_device) for _ in range(2)]

    def step(c, e, ws):
        cu, slots = fa.cache_plan(new, c.cache_len, c.block_table, c.free_blocks, c.free_state, bs, total=B, ws=c.status)
        torch.add(c.cache_len, pre_len, out=e)
        q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
        q = fa.qk_norm_rope_append(q, k, v, c.k, c.v, c.k_scale, c.v_scale, slots, f, cu, ends=e, q_weight=w[0],
                                   k_weight=w[1])
        return fa.forward_paged_prefix(q, c.k, c.v, c.k_scale, c.v_scale, cu, c.cache_len, c.block_table, pcu, plen,
                                       ptable, 1, ws=ws)

    saved = [x.clone() for x in (caches[0].cache_len, caches[0].block_table, caches[0].free_blocks,
                                 caches[0].free_state)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(caches[0], ends[0], ws[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step(caches[0], ends[0], ws[0])
    for x, y in zip((caches[0].cache_len, caches[0].block_table, caches[0].free_blocks, caches[0].free_state), saved):
        x.copy_(y)
    for x in steps:
        qkv.copy_(x)
        graph.replay()
        po, pl = step(caches[1], ends[1], ws[1])
        assert torch.equal(o, po) and torch.equal(lse, pl)
    for c in caches:
        assert fa.get_status(c.status) == fb.FA_OK
    # each request by itself, as one row against the same prefix, within a half step of bf16 of its largest value
    c = caches[1]
    q, k, _ = qkv.split([Hq, Hkv, Hkv], 1)
    q, _ = fa.qk_norm_rope(q, k, f, q_weight=w[0], k_weight=w[1], ends=ends[1],
                           cu_seqlens=torch.arange(B + 1, dtype=torch.int32, device=cuda_device))
    one = dev_i32([0, 1], cuda_device)
    for b in range(B):
        x, _ = fa.forward_paged_prefix(q[b:b + 1].contiguous(), c.k, c.v, c.k_scale, c.v_scale, one,
                                       c.cache_len[b:b + 1].contiguous(), c.block_table[b:b + 1].contiguous(), one,
                                       plen, ptable, 1)
        assert torch.allclose(x[0].float(), po[b].float(), rtol=0, atol=2.0 ** -7 * float(po[b].abs().max()))
