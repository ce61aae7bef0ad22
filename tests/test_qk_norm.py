"""GPU checks of the per-head norm with rotation, its gradient and its cached
form against the fp64 oracle."""

import numpy as np
import pytest
import torch

import io_aware_exact_tiled_gb300 as fa
from io_aware_exact_tiled_gb300 import binding as fb
from oracle import paged as P
from oracle import qk_norm as N

pytestmark = pytest.mark.gpu

EPS = 1e-6
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step of the output's type

# Bounds, in units of 2^-24 of the magnitudes that an element is made of.
# Forward: the sum of squares (8 products a lane in each of two chains, their sum
# and three shuffles: 12 roundings, halved by the root), mean and eps (2, halved),
# rsqrt (2 ulp: 4), two products, cosine and sine (x rounded twice, the series: 4),
# the rotation (2): 19, 32 taken. Backward: the rotated gradient (6), xh (14), the
# product with w (1), the mean of products (21 for its factors, 16 for its sums, 1),
# r (9), the difference and the product (2): 70, 96 taken.
FWD, BWD = 32 * 2.0 ** -24, 96 * 2.0 ** -24


def freqs(rot, theta=1e4):
    return theta ** (-np.arange(0, rot, 2) / rot)


def dev(x, device, dtype=None):
    return torch.tensor(np.asarray(x), dtype=dtype, device=device)


def np64(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Inputs in one of the layouts, with the oracle's view of them."""

    def __init__(self, device, layout, d, rot, Hq, Hkv, inter, norms, dtype, lens=(5, 0, 1, 17), ends=None, seed=0,
                 scale=3.0, theta=1e4):
        rng = np.random.default_rng(seed + d + rot)
        self.d, self.H, self.dtype, self.inter = d, {"q": Hq, "k": Hkv}, dtype, inter
        self.dense = layout == "dense"
        # q, k and something else side by side, as a projection leaves them
        shape = (2, max(lens), Hq + 2 * Hkv, d) if self.dense else (sum(lens) + 3, Hq + 2 * Hkv, d)
        self.qkv = dev(rng.normal(size=shape) * scale, device, dtype)
        self.up = dev(rng.normal(size=shape), device, dtype)
        f = freqs(rot, theta)
        self.f = f
        self.kw = dict(inv_freq=dev(f, device, torch.float64), eps=EPS, interleaved=inter)
        self.w = {}
        for c in "qk":
            self.w[c] = dev(1 + 0.3 * rng.normal(size=d), device, dtype) if c in norms else None
            self.kw[f"{c}_weight"] = self.w[c]
        if self.dense:
            self.pos, self.there = N.positions(shape[1], None, None if ends is None else ends[0])
            if ends is not None:
                self.kw["ends"] = dev([ends[0]] * 2, device, torch.int32)
        else:
            cu = np.concatenate([[2], 2 + np.cumsum(lens)])     # two tokens in front of the first sequence, one behind
            self.kw["cu_seqlens"] = dev(cu, device, torch.int32)
            if ends is not None:
                self.kw["ends"] = dev(ends, device, torch.int32)
            self.pos, self.there = N.positions(shape[0], cu, ends)

    def split(self, t):
        parts = t.split([self.H["q"], self.H["k"], self.H["k"]], -2)
        return {c: x.transpose(1, 2) if self.dense else x for c, x in zip("qkv", parts)}

    def tokens(self, x):
        """[tokens, H, d] in fp64, positions and which tokens are of a sequence."""
        x = np64(x)
        if self.dense:
            b = x.shape[0]
            return x.transpose(0, 2, 1, 3).reshape(-1, x.shape[1], self.d), np.tile(self.pos, b), np.tile(self.there, b)
        return x, self.pos, self.there

    def forward(self, **out):
        x = self.split(self.qkv)
        return dict(zip("qk", fa.qk_norm_rope(x["q"], x["k"], **self.kw, **out)))

    def check_forward(self, got, untouched=None):
        x = self.split(self.qkv)
        for c in "qk":
            y, pos, there = self.tokens(x[c])
            z, m = N.forward(y[there], pos[there], None if self.w[c] is None else np64(self.w[c]), EPS, self.f,
                             self.inter)
            g = self.tokens(got[c])[0]
            err, tol = np.abs(g[there] - z), HALF[self.dtype] * np.abs(z) * (1 + 2.0 ** -8) + FWD * m
            assert (err <= tol).all(), (c, (err / tol).max())
            if untouched is not None:
                assert (g[~there] == untouched).all()

    def check_backward(self, got, dw):
        x, up = self.split(self.qkv), self.split(self.up)
        for c in "qk":
            y, pos, there = self.tokens(x[c])
            u = self.tokens(up[c])[0]
            dx, w, mx, mw = N.backward(y[there], u[there], pos[there],
                                       None if self.w[c] is None else np64(self.w[c]), EPS, self.f, self.inter)
            g = self.tokens(got[c])[0]
            err, tol = np.abs(g[there] - dx), HALF[self.dtype] * np.abs(dx) * (1 + 2.0 ** -8) + BWD * mx
            assert (err <= tol).all(), (c, (err / tol).max())
            if w is None:
                assert dw[c] is None
            else:
                # 20 for a term; its sum: at most one rounding for each row, and 20 for the lanes and CTAs
                tol = (40 + there.sum() * self.H[c]) * 2.0 ** -24 * mw
                err = np.abs(np64(dw[c]) - w)
                assert (err <= tol).all(), (c, (err / tol).max())


SHAPES = [(64, 64, 4, 2), (64, 16, 3, 1), (64, 32, 9, 8), (128, 128, 4, 4), (128, 16, 1, 5), (128, 64, 7, 1),
          (128, 112, 2, 3)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot,Hq,Hkv", SHAPES)
@pytest.mark.parametrize("layout,norms", [("dense", "qk"), ("packed", "qk"), ("packed", "k"), ("dense", "")])
def test_forward_and_backward(cuda_device, layout, norms, d, rot, Hq, Hkv, inter, dtype):
    c = Case(cuda_device, layout, d, rot, Hq, Hkv, inter, norms, dtype)
    x, up = c.split(c.qkv), c.split(c.up)
    out = {k + "_out": torch.full_like(x[k], 7.0) for k in "qk"}
    before = c.qkv.clone()
    c.check_forward(c.forward(**out), untouched=7.0)
    assert torch.equal(c.qkv, before)
    # into the gradient of the projection, whose other part and whose tokens of no sequence stay
    dqkv = torch.full_like(c.qkv, 5.0)
    dx = c.split(dqkv)
    ws = fa.workspace(fa.qk_norm_rope_bwd_workspace_size(d), cuda_device).fill_(255)
    dq, dk, dqw, dkw = fa.qk_norm_rope_backward(x["q"], x["k"], up["q"], up["k"], **c.kw, dq=dx["q"], dk=dx["k"], ws=ws)
    assert fa.get_status(ws) == fb.FA_OK
    assert dq is dx["q"] and dk is dx["k"]
    c.check_backward(dx, {"q": dqw, "k": dkw})
    assert (dx["v"] == 5).all()
    if not c.dense:
        gone = ~torch.tensor(c.there, device=cuda_device)
        assert (dqkv[gone] == 5).all()


@pytest.mark.parametrize("layout", ["dense", "packed"])
def test_positions_from_the_ends(cuda_device, layout):
    """Positions that count back from an end: far ones, negative ones, and the
    last that 32 bits hold."""
    for i, ends in enumerate([(4096, 7, 131072, 9), (2 ** 31 - 1, 0, 3, -5), (12, 2, 1, 2 ** 31 - 1)]):
        c = Case(cuda_device, layout, 128, 128, 3, 1, bool(i & 1), "qk", torch.float32, ends=ends, theta=1e6)
        c.check_forward(c.forward())
        x, up = c.split(c.qkv), c.split(c.up)
        dq, dk, dqw, dkw = fa.qk_norm_rope_backward(x["q"], x["k"], up["q"], up["k"], **c.kw)
        c.check_backward({"q": dq, "k": dk}, {"q": dqw, "k": dkw})


def test_frequencies_of_every_size(cuda_device):
    """Frequencies of many turns a position, negative ones, tiny ones and zero."""
    c = Case(cuda_device, "dense", 64, 16, 2, 2, False, "qk", torch.float32, lens=(40,))
    c.f = np.array([1e6 + 0.3, -1.7, 1e-9, 0.0, 1e-300, -1e-30, 6.283185307179586, 1e11 / 3])
    c.kw["inv_freq"] = dev(c.f, cuda_device, torch.float64)
    c.check_forward(c.forward())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place(cuda_device, dtype):
    c = Case(cuda_device, "packed", 128, 64, 5, 2, False, "qk", dtype)
    want = c.forward()
    got = Case(cuda_device, "packed", 128, 64, 5, 2, False, "qk", dtype)
    x = got.split(got.qkv)
    fa.qk_norm_rope(x["q"], x["k"], **got.kw, q_out=x["q"], k_out=x["k"])
    there = torch.tensor(c.there, device=cuda_device)
    for k in "qk":
        assert torch.equal(x[k][there], want[k][there])
        assert torch.equal(x[k][~there], c.split(c.qkv)[k][~there])
    y, up = c.split(c.qkv), c.split(c.up)
    want = fa.qk_norm_rope_backward(y["q"], y["k"], up["q"], up["k"], **c.kw)
    got = fa.qk_norm_rope_backward(y["q"], y["k"], up["q"], up["k"], **c.kw, dq=up["q"], dk=up["k"])
    for a, b in zip(want[:2], got[:2]):
        assert torch.equal(a[there], b[there])
    assert torch.equal(want[2], got[2]) and torch.equal(want[3], got[3])


def test_special_values(cuda_device):
    """Rows of zeros, of huge and tiny values, with an infinity or a NaN, beside
    ordinary ones: each row by itself."""
    c = Case(cuda_device, "dense", 128, 128, 8, 8, False, "qk", torch.float32, lens=(3,))
    x = c.split(c.qkv)
    with torch.no_grad():
        for i, v in enumerate([0.0, 1e30, 3e37, 1e-30]):
            x["q"][:, i] = torch.sign(x["q"][:, i]) * v
    c.check_forward(c.forward())
    up = c.split(c.up)
    dq, dk, dqw, dkw = fa.qk_norm_rope_backward(x["q"], x["k"], up["q"], up["k"], **c.kw)
    y, pos, _ = c.tokens(x["q"])
    dx, _, mx, _ = N.backward(y, c.tokens(up["q"])[0], pos, np64(c.w["q"]), EPS, c.f, False)
    g = c.tokens(dq)[0]
    assert (np.abs(g - dx) <= (2.0 ** -24 * np.abs(dx) + BWD * mx + 1e-44)).all()
    x["q"][0, 4, 1, 5] = float("inf")
    x["q"][1, 5, 2, 70] = float("nan")
    z = c.forward()["q"]
    assert z[0, 4, 1].isnan().any() and z[1, 5, 2].isnan().all()
    z[0, 4, 1] = z[1, 5, 2] = 0
    assert z.isfinite().all()


@pytest.mark.parametrize("layout,lens", [("dense", (1500,)), ("packed", (900, 1, 0, 1300, 77))])
def test_many_rows(cuda_device, layout, lens):
    """Tokens enough for every CTA to take several; the same bits each time."""
    c = Case(cuda_device, layout, 64, 64, 6, 2, True, "qk", torch.bfloat16, lens=lens)
    first = c.forward()
    c.check_forward(first)
    x, up = c.split(c.qkv), c.split(c.up)
    a = fa.qk_norm_rope_backward(x["q"], x["k"], up["q"], up["k"], **c.kw)
    c.check_backward({"q": a[0], "k": a[1]}, {"q": a[2], "k": a[3]})
    there = torch.tensor(c.there, device=cuda_device)
    for _ in range(3):
        b = fa.qk_norm_rope_backward(x["q"], x["k"], up["q"], up["k"], **c.kw)
        for i in range(2):
            assert torch.equal(a[i] if c.dense else a[i][there], b[i] if c.dense else b[i][there])
        assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])


def test_many_sequences(cuda_device):
    lens = np.random.default_rng(3).integers(0, 3, 3000).tolist()
    c = Case(cuda_device, "packed", 64, 16, 1, 1, False, "q", torch.bfloat16, lens=lens,
             ends=np.random.default_rng(4).integers(0, 5000, 3000).tolist())
    c.check_forward(c.forward())


def test_expanded_input_and_no_tokens(cuda_device):
    """The same row for every head (stride 0), and a batch without tokens."""
    x = torch.randn(1, 1, 9, 64, device=cuda_device).to(torch.bfloat16)
    f = dev(freqs(64), cuda_device, torch.float64)
    q, k = fa.qk_norm_rope(x.expand(1, 4, 9, 64), x, f, q_weight=torch.ones(64, device=cuda_device, dtype=x.dtype))
    assert torch.equal(q[:, 0], q[:, 3]) and q.is_contiguous()
    e = torch.empty(0, 2, 64, device=cuda_device)
    cu = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    w = torch.ones(64, device=cuda_device)
    fa.qk_norm_rope(e, e, f, cu_seqlens=cu)
    assert fa.last_launch_count() == 0
    *_, dw, none = fa.qk_norm_rope_backward(e, e, e, e, f, q_weight=w, cu_seqlens=cu,
                                            dq_weight=torch.ones(64, device=cuda_device))
    assert (dw == 0).all() and none is None


# --------------------------------------------------------------------------
# into the cache
# --------------------------------------------------------------------------

def cache_of(rng, nb, H, bs, d, device):
    b = [torch.tensor(rng.integers(0, 127, (nb, H, bs, d)).astype(np.uint8), device=device).view(torch.float8_e4m3fn)
         for _ in range(2)]
    s = [dev(2.0 ** rng.integers(-12, 3, (nb, H)), device, torch.float32) for _ in range(2)]
    return b + s


def same(a, b):
    for x, y in zip(a, b):
        if x.dtype == torch.float8_e4m3fn:
            x, y = x.view(torch.uint8), y.view(torch.uint8)
        assert torch.equal(x, y)


RUNS = {
    "decode": [(c, 1) for c in range(0, 90, 3)], "one": [(5, 1)], "prompts": [(0, 130), (0, 7), (257, 65), (3, 300)],
    "mixed": [(0, 1), (31, 2), (0, 0), (200, 90), (64, 1), (63, 3), (15, 40)],
    "large": [(0, 600), (7, 500), (0, 1), (100, 301)],
}


@pytest.mark.parametrize("d,rot,Hq,Hkv,inter", [(64, 64, 4, 2, False), (64, 32, 3, 5, True), (128, 128, 8, 1, True),
                                                (128, 16, 2, 9, False)])
@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("which", list(RUNS))
def test_append_equals_the_two_calls(cuda_device, which, bs, d, rot, Hq, Hkv, inter):
    """Bit by bit what the norm and the append write one after the other, whose
    own tests are against their definitions."""
    rng = np.random.default_rng(bs + d)
    reqs = RUNS[which]
    lens = np.array([c + n for c, n in reqs])
    news = [n for _, n in reqs]
    cu = np.concatenate([[0], np.cumsum(news)])
    used = -(-lens // bs)
    nb = int(used.sum()) + 2
    perm = rng.permutation(nb)
    start = np.concatenate([[0], np.cumsum(used)])
    slots = np.concatenate([perm[start[i] + np.arange(c, c + n) // bs] * bs + np.arange(c, c + n) % bs
                            for i, (c, n) in enumerate(reqs)] + [[-1, nb * bs]])
    if which == "decode":
        slots[9] = -1                                    # a token of its sequence without a slot
    total = len(slots)                                   # the last two are of no sequence
    qkv = dev(rng.normal(size=(total, Hq + 2 * Hkv, d)) * 2.0 ** rng.integers(-6, 6, (total, 1, 1)), cuda_device,
              torch.bfloat16)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    kw = dict(inv_freq=dev(freqs(rot), cuda_device, torch.float64), eps=EPS, interleaved=inter,
              cu_seqlens=dev(cu, cuda_device, torch.int32), ends=dev(lens + 1000, cuda_device, torch.int32),
              q_weight=dev(rng.normal(size=d), cuda_device, torch.bfloat16),
              k_weight=dev(rng.normal(size=d), cuda_device, torch.bfloat16) if which != "one" else None)
    ids = dev(slots, cuda_device, torch.int32)
    ours = cache_of(rng, nb, Hkv, bs, d, cuda_device)
    theirs = [x.clone() for x in ours]
    out = torch.full((total, Hq, d), 7.0, dtype=torch.bfloat16, device=cuda_device)
    q_out = fa.qk_norm_rope_append(q, k, v, *ours, ids, **kw, q_out=out)
    assert q_out is out and fa.last_launch_count() == (2 if total > 1024 else 1)
    qn, kn = fa.qk_norm_rope(q, k, **kw)
    fa.cache_append(kn, v.contiguous(), *theirs, ids)
    assert torch.equal(q_out[:-2], qn[:-2]) and (q_out[-2:] == 7).all()
    same(ours, theirs)


def test_append_against_the_definition(cuda_device):
    """The whole of it against the oracle: its key in bf16 may be the other
    neighbour, so a stored value is within the key's half step and its own."""
    rng = np.random.default_rng(1)
    d, bs, Hq, Hkv, total = 128, 32, 4, 2, 70
    qkv = dev(rng.normal(size=(total, Hq + 2 * Hkv, d)), cuda_device, torch.bfloat16)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    f = freqs(d)
    w = dev(1 + 0.2 * rng.normal(size=d), cuda_device, torch.bfloat16)
    c = cache_of(rng, 4, Hkv, bs, d, cuda_device)
    slots = np.arange(total) + bs
    fa.qk_norm_rope_append(q, k, v, *c, dev(slots, cuda_device, torch.int32), dev(f, cuda_device, torch.float64),
                           dev([0, total], cuda_device, torch.int32), k_weight=w)
    z, m = N.forward(np64(k), np.arange(total), np64(w), EPS, f, False)
    stored = P.e4m3_decode(c[0].view(torch.uint8).cpu().numpy()) * np64(c[2])[:, :, None, None]
    stored = stored[1:].transpose(0, 2, 1, 3).reshape(-1, Hkv, d)[:total]
    scale = np.repeat(np64(c[2])[1:], bs, 0)[:total][..., None]
    tol = np.abs(z) * (2.0 ** -4 + 2.0 ** -7) + scale * 2.0 ** -10 + FWD * m     # E4M3's half step, 2^-10 below 2^-6
    assert (np.abs(stored - z) <= tol).all()
    want, ws = P.append(np64(v), np.zeros((4, Hkv, bs, d), np.uint8), np.ones((4, Hkv)), slots)
    np.testing.assert_array_equal(c[1].view(torch.uint8).cpu().numpy()[1:3], want[1:3])
    np.testing.assert_array_equal(np64(c[3])[1:], ws[1:])


def test_append_nothing(cuda_device):
    c = fa.paged_cache(2, 1, 16, 64, 1, 2, cuda_device)
    e = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=cuda_device)
    i32 = dict(dtype=torch.int32, device=cuda_device)
    fa.qk_norm_rope_append(e, e, e, c.k, c.v, c.k_scale, c.v_scale, torch.empty(0, **i32),
                           dev(freqs(64), cuda_device, torch.float64), torch.zeros(2, **i32))
    assert fa.last_launch_count() == 0
