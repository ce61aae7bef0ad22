"""`stream=` of the binding's entry points: what a call allocates by itself
belongs to the stream that it runs on."""

import contextlib
import inspect
import types

import pytest
import torch

import io_aware_exact_tiled_gb300 as fa
from io_aware_exact_tiled_gb300 import binding as fb

from test_binding import FakeLib


def calls(dev):
    """Every entry point that takes a stream, with tensors as it wants them and
    no outputs or workspace."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    q = bf(1, 1, 128, 64)
    lse = torch.zeros((1, 1, 128), device=dev)
    x, xl = bf(128, 1, 64), torch.zeros((1, 128), device=dev)
    c = fa.paged_cache(4, 1, 16, 64, 1, 4, dev)
    return {
        "forward": (q, q, q), "backward": (q, q, q, q, lse, q), "backward_noalloc": (q, q, q, q, lse, q),
        "forward_varlen": (x, x, x, i32(0, 128), 128), "backward_varlen": (x, x, x, x, xl, x, i32(0, 128), 128),
        "forward_fp8": (q, q, q, None), "forward_dropout": (q, q, q, 0.1, 1), "backward_dropout": (q, q, q, q, lse, q, 0.1, 1),
        "decode": (bf(1, 1, 1, 64), q, q),
        "cache_plan": (i32(1), c.cache_len, c.block_table, c.free_blocks, c.free_state, 16, 1),
        "cache_append": (bf(1, 1, 64), bf(1, 1, 64), c.k, c.v, c.k_scale, c.v_scale, i32(0)),
        "forward_paged": (bf(1, 1, 64), c.k, c.v, c.k_scale, c.v_scale, i32(0, 1), i32(1), i32(0, -1)[None], 1),
    }


def test_every_stream_argument_is_covered():
    with_stream = {n for n, f in vars(fb).items() if inspect.isfunction(f) and not n.startswith(("_", "fa_"))
                   and "stream" in inspect.signature(f).parameters}
    assert with_stream == set(calls("cpu")) | {"get_status", "noalloc_status"}


@pytest.mark.parametrize("name", list(calls("cpu")))
@pytest.mark.parametrize("positional", [False, True])
def test_buffers_are_allocated_on_the_given_stream(monkeypatch, name, positional):
    lib, now, seen = FakeLib(), [None], []
    args = calls("cpu")
    monkeypatch.setattr(fb, "_lib", lib)
    monkeypatch.setattr(fb, "_check_device", lambda q: None)
    monkeypatch.setattr(fb, "_stream_handle", lambda stream=None: stream or now[0])

    @contextlib.contextmanager
    def on(s):
        now[0] = s
        yield
        now[0] = None

    real = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: seen.append(now[0]) or real(*a, **kw))
    f, a, mine = getattr(fb, name), args[name], 1234
    if positional:
        names = list(inspect.signature(f).parameters)
        assert names[-1] == "stream"
        given = inspect.signature(f).bind(*a, stream=mine)
        given.apply_defaults()
        f(*given.args)
    else:
        f(*a, stream=mine)
    assert set(seen) == {mine} or name == "cache_append" and not seen
    assert lib.calls[-1][1][-1] == mine and now == [None]
    seen.clear()
    f(*a)
    assert set(seen) <= {None} and lib.calls[-1][1][-1] is None


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["forward", "forward_paged"])
def test_outputs_belong_to_the_given_stream(cuda_device, name):
    args = calls(cuda_device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = getattr(fa, name)(*args[name], stream=side)
    side.synchronize()
    owner = {}
    for seg in torch.cuda.memory_snapshot():
        for t in (o, lse):
            if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
                owner[t.data_ptr()] = seg["stream"]
    assert set(owner.values()) == {side.cuda_stream} and len(owner) == 2
    want = getattr(fa, name)(*args[name])
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    other = types.SimpleNamespace(device_index=1, device="cuda:1", cuda_stream=7)
    with pytest.raises(ValueError, match="stream"):
        fb._stream_handle(other)
    other.device_index = 0
    assert fb._stream_handle(other) == 7
