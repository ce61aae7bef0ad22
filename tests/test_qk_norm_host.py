"""Norm with rotation and attention with shared prefixes on the CPU: refusals of
the entry points, workspace sizes, and the binding's argument order and checks."""

import contextlib
import inspect
import struct

import pytest
import torch

import io_aware_exact_tiled_gb300 as fa
from io_aware_exact_tiled_gb300 import binding as fb
from io_aware_exact_tiled_gb300 import build as fbuild
from io_aware_exact_tiled_gb300 import qk_norm

from test_binding import FakeLib, addr, last

FAKE, MIS = 1 << 20, (1 << 20) + 2
OK, BAD, NO = fb.FA_OK, fb.FA_ERR_INVALID_ARG, fb.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fb.load()


def rows(data=FAKE, batch=8 * 64 * 4, head=64, token=4 * 64):
    return qk_norm._pack_rows(data or 0, batch, head, token)


NORM = dict(eps=1e-6, inv_freq=FAKE, rot=64, inter=0, cu=None, ends=None, B=2, N=8, Hq=4, Hkv=4, d=64,
            dtype=fb.FA_BF16)


def norm(lib, r=None, qw=FAKE, kw=FAKE, **over):
    a = NORM | over
    r = [rows()] * 4 if r is None else r
    return lib.fa_qk_norm_rope(*r, qw, kw, a["eps"], a["inv_freq"], a["rot"], a["inter"], a["cu"], a["ends"], a["B"],
                               a["N"], a["Hq"], a["Hkv"], a["d"], a["dtype"], None)


def norm_bwd(lib, r=None, qw=FAKE, kw=FAKE, dqw=FAKE, dkw=FAKE, ws=FAKE, wsb=1 << 30, **over):
    a = NORM | over
    r = [rows()] * 6 if r is None else r
    return lib.fa_qk_norm_rope_bwd(*r, qw, kw, dqw, dkw, a["eps"], a["inv_freq"], a["rot"], a["inter"], a["cu"],
                                   a["ends"], a["B"], a["N"], a["Hq"], a["Hkv"], a["d"], a["dtype"], ws, wsb, None)


SIZES = [(dict(B=0), BAD), (dict(N=-1), BAD), (dict(Hq=0), BAD), (dict(Hkv=-2), BAD), (dict(d=0), BAD),
         (dict(rot=0), BAD), (dict(eps=0.0), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
         (dict(eps=float("inf")), BAD), (dict(inter=2), BAD), (dict(dtype=5), BAD), (dict(inv_freq=None), BAD),
         (dict(inv_freq=FAKE + 4), BAD), (dict(ends=MIS), BAD), (dict(cu=MIS), BAD), (dict(d=96, rot=32), NO),
         (dict(d=256), NO), (dict(rot=8), NO), (dict(rot=80), NO), (dict(rot=24), NO), (dict(Hq=1 << 16), NO),
         (dict(B=1 << 16, cu=FAKE), NO), (dict(B=1 << 15, N=1 << 14), NO)]
ROWS = [None, rows(data=None), rows(data=FAKE + 8), rows(batch=-8), rows(token=4), rows(head=12),
        rows(batch=(1 << 62))]
OVERLAPS = [rows(token=32), rows(head=0), rows(batch=0), rows(batch=64 * 4), rows(head=64, token=128)]


def test_norm_refusals(lib):
    for over, code in SIZES:
        assert norm(lib, **over) == code, over
        assert norm_bwd(lib, **over) == code, over
    for i in range(4):
        for bad in ROWS + (OVERLAPS if i >= 2 else []):
            assert norm(lib, r=[bad if x == i else rows() for x in range(4)]) == BAD, (i, bad)
    for i in range(6):
        for bad in ROWS + (OVERLAPS if i >= 4 else []):
            assert norm_bwd(lib, r=[bad if x == i else rows() for x in range(6)]) == BAD, (i, bad)
    assert norm(lib, qw=MIS) == BAD and norm(lib, kw=MIS) == BAD
    for kw in (dict(qw=None), dict(kw=None), dict(dqw=None), dict(dkw=None), dict(dqw=MIS), dict(ws=None),
               dict(ws=FAKE + 16), dict(wsb=4096)):
        assert norm_bwd(lib, **kw) == BAD, kw
    # fp32 rows need strides of four elements, bf16 ones of eight
    assert norm(lib, r=[rows(token=4 * 64 + 4)] + [rows()] * 3) == BAD
    # no tokens: nothing to do, whatever the rows are
    assert norm(lib, r=[None] * 4, N=0) == OK and lib.fa_last_launch_count() == 0
    assert lib.fa_qk_norm_rope_bwd_workspace_size(0) == 0
    assert lib.fa_qk_norm_rope_bwd_workspace_size(128) >= 256 + 2 * 128 * 4


def append(lib, r=None, ptrs=None, cu=FAKE, bs=16, nb=64, **over):
    a = NORM | dict(N=8) | over
    p = [FAKE] * 5
    for i, v in (ptrs or {}).items():
        p[i] = v
    r = [rows()] * 4 if r is None else r
    return lib.fa_qk_norm_rope_append(*r, *p, FAKE, FAKE, a["eps"], a["inv_freq"], a["rot"], a["inter"], cu, a["ends"],
                                      a["B"], a["N"], a["Hq"], a["Hkv"], a["d"], nb, bs, None)


def test_append_refusals(lib):
    for over, code in SIZES:
        if "cu" not in over and "dtype" not in over and over != dict(B=1 << 15, N=1 << 14):
            assert append(lib, **over) == code, over
    for i in range(5):
        assert append(lib, ptrs={i: None}) == BAD and append(lib, ptrs={i: MIS}) == BAD, i
    assert append(lib, cu=None) == BAD and append(lib, cu=MIS) == BAD
    for i in range(4):
        for bad in [x for x in ROWS if x is None or row(x)[1] == 8 * 64 * 4] + (OVERLAPS[:2] if i == 3 else []):
            assert append(lib, r=[bad if x == i else rows() for x in range(4)]) == BAD, (i, bad)
    for kw in (dict(bs=8), dict(bs=48), dict(bs=512), dict(nb=1 << 26)):
        assert append(lib, **kw) == NO, kw
    assert append(lib, bs=0) == BAD and append(lib, nb=0) == BAD
    assert append(lib, r=[None] * 4, ptrs={4: None}, N=0) == OK and lib.fa_last_launch_count() == 0


def prefix(lib, ptrs=None, B=4, P=2, Hq=4, Hkv=2, total=8, max_new=4, mb=8, pb=8, nb=64, bs=16, d=64, scale=0.1,
           causal=1, ws=FAKE, wsb=1 << 40):
    p = [FAKE] * 13
    for i, v in (ptrs or {}).items():
        p[i] = v
    return lib.fa_fwd_paged_prefix(*p, B, P, Hq, Hkv, total, max_new, mb, pb, nb, bs, d, scale, causal, ws, wsb, None)


def test_prefix_refusals(lib):
    for i in range(13):
        assert prefix(lib, {i: None}) == BAD and prefix(lib, {i: MIS}) == BAD, i
    assert prefix(lib, ws=None) == BAD and prefix(lib, ws=FAKE + 16) == BAD and prefix(lib, wsb=1024) == BAD
    for kw in (dict(B=0), dict(P=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(total=-1), dict(max_new=-1),
               dict(max_new=9), dict(mb=0), dict(pb=0), dict(nb=0), dict(bs=0), dict(d=0), dict(causal=2),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0)):
        assert prefix(lib, **kw) == BAD, kw
    for kw in (dict(d=96), dict(bs=24), dict(B=1 << 16), dict(P=1 << 16), dict(Hq=1 << 16), dict(mb=1 << 27),
               dict(pb=1 << 27), dict(nb=1 << 27), dict(total=1 << 30)):
        assert prefix(lib, **kw) == NO, kw


def test_prefix_workspace_size(lib):
    size = lib.fa_fwd_paged_prefix_workspace_size
    for bad in ((0, 1, 4, 2, 8, 1, 64), (1, 0, 4, 2, 8, 1, 64), (1, 1, 3, 2, 8, 1, 64), (1, 1, 4, 2, -1, 1, 64)):
        assert size(*bad) == 0
    # what the prefixes' pass leaves, and the workspaces of both passes
    one = size(4, 1, 4, 2, 8, 1, 64)
    assert one >= 8 * 4 * (64 + 2) * 4 + 2 * (lib.fa_fwd_paged_workspace_size(4, 4, 2, 8, 1, 64) - 2048)
    assert size(4, 1, 4, 2, 8, 8, 64) >= one and prefix(lib, P=1, max_new=1, wsb=one - 1) == BAD


# --------------------------------------------------------------------------
# binding
# --------------------------------------------------------------------------

@pytest.fixture
def fake(monkeypatch):
    fake = FakeLib()
    monkeypatch.setattr(fb, "_lib", fake)
    monkeypatch.setattr(fb, "_check_device", lambda q: None)
    monkeypatch.setattr(fb, "_stream_handle", lambda stream=None: None)
    return fake


def row(a):
    return struct.unpack("@Pqqq", a)


def test_norm_argument_order(fake):
    B, N, Hq, Hkv, d = 2, 5, 3, 1, 64
    qkv = torch.zeros(B, N, Hq + 2 * Hkv, d, dtype=torch.bfloat16)
    q, k, _ = (x.transpose(1, 2) for x in qkv.split([Hq, Hkv, Hkv], 2))
    w, f = torch.ones(d, dtype=torch.bfloat16), torch.ones(16, dtype=torch.float64)
    ends = torch.zeros(B, dtype=torch.int32)
    q_out, k_out = fa.qk_norm_rope(q, k, f, q_weight=w, ends=ends, eps=0.5, interleaved=True)
    a = last(fake, "fa_qk_norm_rope")
    assert row(a[0]) == (addr(q), N * 5 * d, d, 5 * d) and row(a[1])[0] == addr(k)
    assert row(a[2]) == (addr(q_out), Hq * N * d, N * d, d) and row(a[3])[0] == addr(k_out)
    assert a[4:] == [addr(w), None, 0.5, addr(f), 32, 1, None, addr(ends), B, N, Hq, Hkv, d, fb.FA_BF16, None]
    dq, dk, dqw, dkw = fa.qk_norm_rope_backward(q, k, q_out, k_out, f, q_weight=w)
    a = last(fake, "fa_qk_norm_rope_bwd")
    assert [row(x)[0] for x in a[:6]] == [addr(x) for x in (q, k, q_out, k_out, dq, dk)]
    assert a[6:10] == [addr(w), None, addr(dqw), None] and dkw is None and dqw.dtype == torch.float32
    assert a[10:22] == [1e-6, addr(f), 32, 0, None, None, B, N, Hq, Hkv, d, fb.FA_BF16] and a[23] == 4096
    # packed
    x = torch.zeros(7, 4, d)
    q, k = x[:, :3], x[:, 3:]
    cu = torch.zeros(3, dtype=torch.int32)
    fa.qk_norm_rope(q, k, f, cu_seqlens=cu, q_out=q, k_out=k)
    a = last(fake, "fa_qk_norm_rope")
    assert row(a[0]) == (addr(q), 0, d, 4 * d) == row(a[2]) and a[10] == addr(cu)
    assert a[12:18] == [2, 7, 3, 1, d, fb.FA_FP32]


def test_append_and_prefix_argument_order(fake):
    total, Hq, Hkv, d, nb, bs, B, P = 6, 4, 2, 64, 9, 16, 3, 2
    q, k, v = torch.zeros(total, Hq + 2 * Hkv, d, dtype=torch.bfloat16).split([Hq, Hkv, Hkv], 1)
    c = fb.paged_cache(nb, Hkv, bs, d, B, 4, "cpu")
    f, w = torch.ones(32, dtype=torch.float64), torch.ones(d, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    cu, slots, ends = torch.zeros(B + 1, **i32), torch.zeros(total, **i32), torch.zeros(B, **i32)
    o = fa.qk_norm_rope_append(q, k, v, c.k, c.v, c.k_scale, c.v_scale, slots, f, cu, ends=ends, k_weight=w)
    a = last(fake, "fa_qk_norm_rope_append")
    assert [row(x)[0] for x in a[:4]] == [addr(x) for x in (q, k, v, o)]
    assert a[4:9] == [addr(x) for x in (c.k, c.v, c.k_scale, c.v_scale, slots)] and a[9:11] == [None, addr(w)]
    assert a[11:] == [1e-6, addr(f), 64, 0, addr(cu), addr(ends), B, total, Hq, Hkv, d, nb, bs, None]
    pcu, plen, ptab = torch.zeros(P + 1, **i32), torch.zeros(P, **i32), torch.zeros(P, 5, **i32)
    y, L = fa.forward_paged_prefix(o, c.k, c.v, c.k_scale, c.v_scale, cu, c.cache_len, c.block_table, pcu, plen, ptab,
                                   4, scale=0.5)
    a = last(fake, "fa_fwd_paged_prefix")
    assert a[:13] == [addr(x) for x in (o, c.k, c.v, c.k_scale, c.v_scale, y, L, cu, c.cache_len, c.block_table, pcu,
                                        plen, ptab)]
    assert a[13:24] == [B, P, Hq, Hkv, total, 4, 4, 5, nb, bs, d] and a[24:26] == [0.5, 1] and a[27] == 4096
    assert last(fake, "fa_fwd_paged_prefix_workspace_size") == [B, P, Hq, Hkv, total, 4, d]
    i = len(fake.calls)
    for bad in (dict(prefix_cu=pcu[:2]), dict(prefix_len=plen.long()), dict(prefix_table=ptab[0]),
                dict(prefix_table=ptab.t()), dict(out=y[:3]), dict(cache_len=cu)):
        kw = dict(prefix_cu=pcu, prefix_len=plen, prefix_table=ptab, cache_len=c.cache_len) | bad
        with pytest.raises(ValueError):
            fa.forward_paged_prefix(o, c.k, c.v, c.k_scale, c.v_scale, cu, block_table=c.block_table, max_new=4, **kw)
    for bad in (dict(cu_seqlens=None), dict(slots=slots[:2]), dict(v=v[:, :1]), dict(q=q.float()), dict(ends=cu),
                dict(k=k[:, :1], v=v[:, :1])):
        kw = dict(q=q, k=k, v=v, slots=slots, inv_freq=f, cu_seqlens=cu) | bad
        with pytest.raises(ValueError):
            fa.qk_norm_rope_append(k_cache=c.k, v_cache=c.v, k_scale=c.k_scale, v_scale=c.v_scale, **kw)
    assert len(fake.calls) == i


def test_wrong_norm_tensors_are_refused_before_the_call(fake):
    q, k = torch.zeros(2, 3, 5, 64), torch.zeros(2, 1, 5, 64)
    f, w = torch.ones(32, dtype=torch.float64), torch.ones(64)
    cu = torch.zeros(3, dtype=torch.int32)
    for bad in (dict(k=k[:1]), dict(k=k[..., :32]), dict(k=k.bfloat16()), dict(k=k[0]), dict(q=q.half(), k=k.half()),
                dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), dict(inv_freq=f.float()),
                dict(inv_freq=f[None]), dict(inv_freq=f[::2]), dict(q_weight=w[:32]), dict(k_weight=w.bfloat16()),
                dict(cu_seqlens=cu), dict(ends=cu), dict(ends=cu[:2].long()), dict(q_out=q[:, :2]),
                dict(k_out=k.bfloat16()), dict(q=q[0], k=k[0])):
        with pytest.raises(ValueError):
            fa.qk_norm_rope(**(dict(q=q, k=k, inv_freq=f) | bad))
        up = {f"d{c}_out": torch.zeros_like((dict(q=q, k=k) | bad)[c]) for c in "qk"}
        bad = {("d" + c[0] if c in ("q_out", "k_out") else c): x for c, x in bad.items()}
        with pytest.raises(ValueError):
            fa.qk_norm_rope_backward(**(dict(q=q, k=k, inv_freq=f) | up | bad))
    with pytest.raises(ValueError):
        fa.qk_norm_rope_backward(q, k, q, k, f, dq_weight=w)
    assert not [c for c in fake.calls if not c[0].endswith("_workspace_size")]


def stream_calls():
    """The calls that take a stream, with no outputs or workspace."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    q, f, w = bf(1, 1, 4, 64), torch.ones(32, dtype=torch.float64), bf(64)
    x, c = bf(1, 1, 64), fb.paged_cache(4, 1, 16, 64, 1, 4, "cpu")
    return {"qk_norm_rope": (q, q, f, w, w), "qk_norm_rope_backward": (q, q, q, q, f, w, w),
            "qk_norm_rope_append": (x, x, x, c.k, c.v, c.k_scale, c.v_scale, i32(0), f, i32(0, 1)),
            "forward_paged_prefix": (x, c.k, c.v, c.k_scale, c.v_scale, i32(0, 1), i32(1), i32(0, -1)[None], i32(0, 1),
                                     i32(3), i32(1)[None], 1)}


@pytest.mark.parametrize("name", list(stream_calls()))
def test_buffers_are_allocated_on_the_given_stream(monkeypatch, fake, name):
    now, seen = [None], []
    args = stream_calls()[name]
    monkeypatch.setattr(fb, "_stream_handle", lambda stream=None: stream or now[0])

    @contextlib.contextmanager
    def on(s):
        now[0] = s
        yield
        now[0] = None

    real = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: seen.append(now[0]) or real(*a, **kw))
    f, mine = getattr(fa, name), 1234
    assert list(inspect.signature(f).parameters)[-1] == "stream"
    f(*args, stream=mine)
    assert set(seen) == {mine} and fake.calls[-1][1][-1] == mine and now == [None]
    seen.clear()
    f(*args)
    assert set(seen) == {None} and fake.calls[-1][1][-1] is None
