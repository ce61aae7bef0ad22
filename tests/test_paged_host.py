"""Paged cache on the CPU: every refusal of the three entry points, their
workspace size, and the binding's argument order and checks."""

import ctypes

import pytest
import torch

from io_aware_exact_tiled_gb300 import binding as fb
from io_aware_exact_tiled_gb300 import build as fbuild

from test_binding import FakeLib, addr, last

FAKE, MIS = 1 << 20, (1 << 20) + 2
OK, BAD, NO = fb.FA_OK, fb.FA_ERR_INVALID_ARG, fb.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fb.load()


def plan(lib, ptrs=None, B=4, max_blocks=8, num_blocks=64, bs=16, total=4, wsb=256):
    p = [FAKE] * 9
    for i, v in (ptrs or {}).items():
        p[i] = v
    ws = p.pop() if len(p) > 9 else FAKE
    return lib.fa_cache_plan(*p, B, max_blocks, num_blocks, bs, total, ws, wsb, None)


def test_plan_refusals(lib):
    for i in range(9):
        assert plan(lib, {i: None}) == BAD, i
        assert plan(lib, {i: MIS}) == BAD, i
    assert plan(lib, wsb=128) == BAD
    for kw in (dict(B=0), dict(max_blocks=0), dict(num_blocks=-1), dict(bs=0), dict(total=-1)):
        assert plan(lib, **kw) == BAD, kw
    for kw in (dict(bs=8), dict(bs=24), dict(bs=512), dict(B=16385), dict(total=(1 << 30) + 1),
               dict(max_blocks=1 << 27), dict(num_blocks=1 << 27)):
        assert plan(lib, **kw) == NO, kw


def append(lib, ptrs=None, total=4, H=2, d=64, num_blocks=64, bs=16):
    p = [FAKE] * 7
    for i, v in (ptrs or {}).items():
        p[i] = v
    return lib.fa_cache_append(*p, total, H, d, num_blocks, bs, None)


def test_append_refusals(lib):
    for i in range(7):
        assert append(lib, {i: None}) == BAD, i
        assert append(lib, {i: MIS}) == BAD, i
    assert append(lib, {0: FAKE + 8}) == BAD and append(lib, {2: FAKE + 4}) == BAD
    for kw in (dict(total=-1), dict(H=0), dict(d=0), dict(num_blocks=0), dict(bs=-16)):
        assert append(lib, **kw) == BAD, kw
    for kw in (dict(d=96), dict(d=256), dict(bs=48), dict(num_blocks=1 << 25, H=8), dict(total=1 << 30, H=2)):
        assert append(lib, **kw) == NO, kw
    # no tokens: nothing to do, whatever the token pointers are
    assert append(lib, {0: None, 1: None, 6: None}, total=0) == OK
    assert lib.fa_last_launch_count() == 0


def fwd(lib, ptrs=None, B=2, Hq=4, Hkv=2, total=8, max_new=4, max_blocks=8, num_blocks=64, bs=16, d=64, scale=0.1,
        causal=1, ws=FAKE, wsb=1 << 30):
    p = [FAKE] * 10
    for i, v in (ptrs or {}).items():
        p[i] = v
    return lib.fa_fwd_paged(*p, B, Hq, Hkv, total, max_new, max_blocks, num_blocks, bs, d, scale, causal, ws, wsb, None)


def test_fwd_refusals(lib):
    for i in range(10):
        assert fwd(lib, {i: None}) == BAD, i
        assert fwd(lib, {i: MIS}) == BAD, i
    assert fwd(lib, ws=None) == BAD and fwd(lib, ws=FAKE + 16) == BAD and fwd(lib, wsb=1024) == BAD
    for kw in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(total=-1), dict(max_new=-1), dict(max_new=9),
               dict(max_blocks=0), dict(num_blocks=0), dict(bs=0), dict(d=0), dict(causal=2), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1.0)):
        assert fwd(lib, **kw) == BAD, kw
    for kw in (dict(d=80), dict(d=256), dict(bs=8), dict(bs=512), dict(B=65536), dict(Hq=65536, Hkv=65536),
               dict(total=1 << 30), dict(max_blocks=1 << 27), dict(num_blocks=1 << 26)):
        assert fwd(lib, **kw) == NO, kw


def test_workspace_size(lib):
    size = lib.fa_fwd_paged_workspace_size
    assert size(0, 4, 2, 8, 1, 64) == 0 and size(2, 3, 2, 8, 1, 64) == 0 and size(2, 4, 2, -1, 1, 64) == 0
    few, many = size(2, 4, 2, 8, 4, 64), size(2, 4, 2, 80, 40, 64)
    assert few >= 256 + 304 * 32 * 64 * 4                 # partial outputs of up to 32 rows
    assert many - few >= 304 * 256 * 64 * 4               # requests of more than 32 rows: 256-row partials too
    assert size(2, 4, 2, 80, 16, 64) <= few + 1024        # 16 tokens of two heads a group: 32 rows
    # it is what the call asks for
    assert fwd(lib, wsb=few - 1) == BAD
    # it grows with the requests, the tokens and the head size
    assert size(5000, 4, 2, 8, 4, 64) > few and size(2, 4, 2, 8, 4, 128) > few and size(2, 4, 2, 1 << 20, 40, 64) > many


def test_status_code_for_a_free_list_that_ran_out(lib):
    assert fb.status_string(fb.FA_ERR_NO_BLOCKS).startswith("FA_ERR_NO_BLOCKS")


@pytest.fixture
def fake(monkeypatch):
    f = FakeLib()
    monkeypatch.setattr(fb, "_lib", f)
    monkeypatch.setattr(fb, "_check_device", lambda q: None)
    monkeypatch.setattr(fb, "_stream_handle", lambda stream=None: None)
    return f


def test_binding_argument_order(fake):
    c = fb.paged_cache(10, 2, 32, 64, 3, 4, device="cpu")
    assert c.k.dtype == torch.float8_e4m3fn and c.k.shape == (10, 2, 32, 64) and c.free_state.tolist() == [0, 10]
    new = torch.ones(3, dtype=torch.int32)
    ws = torch.empty(256, dtype=torch.uint8)
    cu, slots = fb.cache_plan(new, c.cache_len, c.block_table, c.free_blocks, c.free_state, 32, total=3, ws=ws)
    a = last(fake, "fa_cache_plan")
    assert a[:9] == [addr(t) for t in (new, c.cache_len, c.cache_len, c.block_table, c.free_blocks, c.free_state,
                                       c.free_state, cu, slots)]
    assert a[9:16] == [3, 4, 10, 32, 3, addr(ws), 256] and cu.shape == (4,) and slots.shape == (3,)
    out, state = torch.empty_like(c.cache_len), torch.empty_like(c.free_state)
    fb.cache_plan(new, c.cache_len, c.block_table, c.free_blocks, c.free_state, 32, slots=slots, cache_len_out=out,
                  free_state_out=state)
    a = last(fake, "fa_cache_plan")
    assert a[1:3] == [addr(c.cache_len), addr(out)] and a[5:7] == [addr(c.free_state), addr(state)] and a[13] == 3

    k, v = (torch.zeros(3, 2, 64, dtype=torch.bfloat16) for _ in range(2))
    fb.cache_append(k, v, c.k, c.v, c.k_scale, c.v_scale, slots)
    a = last(fake, "fa_cache_append")
    assert a[:7] == [addr(t) for t in (k, v, c.k, c.v, c.k_scale, c.v_scale, slots)] and a[7:12] == [3, 2, 64, 10, 32]

    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    o, lse = fb.forward_paged(q, c.k, c.v, c.k_scale, c.v_scale, cu, c.cache_len, c.block_table, 1, scale=0.5,
                              causal=False)
    a = last(fake, "fa_fwd_paged")
    assert a[:10] == [addr(t) for t in (q, c.k, c.v, c.k_scale, c.v_scale, o, lse, cu, c.cache_len, c.block_table)]
    assert a[10:21] == [3, 8, 2, 3, 1, 4, 10, 32, 64, 0.5, 0] and a[22] == 4096 and lse.shape == (8, 3)
    assert last(fake, "fa_fwd_paged_workspace_size") == [3, 8, 2, 3, 1, 64]
    fb.fa_fwd_paged_workspace_size(1, 2, 1, 4, 5, 128)
    assert last(fake, "fa_fwd_paged_workspace_size") == [1, 2, 1, 4, 5, 128]


def test_binding_refuses_before_the_call(fake):
    c = fb.paged_cache(10, 2, 32, 64, 3, 4, device="cpu")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    plan_args = [i32(3), c.cache_len, c.block_table, c.free_blocks, c.free_state, 32]
    for i, bad in ((0, i32(2)), (0, i32(3, 1)), (1, torch.zeros(3, dtype=torch.int64)), (2, i32(4, 4)), (2, i32(4)),
                   (3, i32(20)[::2]), (4, i32(3))):
        args = list(plan_args)
        args[i] = bad
        with pytest.raises(ValueError):
            fb.cache_plan(*args, total=3)
    with pytest.raises(ValueError, match="total"):
        fb.cache_plan(*plan_args)
    for kw in (dict(slots=i32(4), total=3), dict(cu_seqlens=i32(3), total=3), dict(cache_len_out=i32(2), total=3),
               dict(free_state_out=i32(3), total=3)):
        with pytest.raises(ValueError):
            fb.cache_plan(*plan_args, **kw)
    for bad in (dict(k=k.float()), dict(v=k[:2]), dict(k_cache=c.k.view(torch.uint8)), dict(k_cache=c.k[:, :1]),
                dict(v_cache=c.v[:9]), dict(k_scale=c.k_scale.double()), dict(v_scale=c.v_scale[:, :1]),
                dict(slots=i32(2)), dict(k=torch.zeros(3, 2, 128, dtype=torch.bfloat16))):
        args = dict(k=k, v=k, k_cache=c.k, v_cache=c.v, k_scale=c.k_scale, v_scale=c.v_scale, slots=i32(3)) | bad
        with pytest.raises(ValueError):
            fb.cache_append(**args)
    for bad in (dict(q=q.half()), dict(q=q[:, :, :32]), dict(q=q.transpose(0, 1)), dict(cu_seqlens=i32(3)),
                dict(cache_len=i32(4)), dict(block_table=i32(3, 8)[:, ::2]), dict(k_cache=c.k[0]),
                dict(out=q.float()), dict(lse=torch.zeros(3, 8)), dict(ws=torch.zeros(8, 64)[:, ::2])):
        args = dict(q=q, k_cache=c.k, v_cache=c.v, k_scale=c.k_scale, v_scale=c.v_scale, cu_seqlens=i32(4),
                    cache_len=i32(3), block_table=c.block_table, max_new=1) | bad
        with pytest.raises(ValueError):
            fb.forward_paged(**args)
    assert fake.calls == []


def test_tensors_must_be_on_the_current_cuda_device():
    c = fb.paged_cache(2, 1, 16, 64, 1, 2, device="cpu")
    k = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fb.cache_append(k, k, c.k, c.v, c.k_scale, c.v_scale, torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("d", list(range(1, 70)) + [71, 127, 128, 255, 1000, 4095, 65535])
def test_division_by_multiplication(d):
    """The quotient that the kernels form for the heads of a group, restated."""
    l = (d - 1).bit_length()
    m = (((1 << l) - d) << 32) // d + 1
    assert m < 1 << 32
    xs = set(range(0, 300)) | {(1 << 31) - 1 - i for i in range(5)}
    for q in (1, 2, 1000, ((1 << 31) - 1) // d):
        xs |= {q * d - 1, q * d, q * d + 1}
    for x in xs:
        if 0 <= x < 1 << 31:
            hi = (m * x) >> 32
            assert hi + x < 1 << 32 and (hi + x) >> l == x // d, (x, d)
