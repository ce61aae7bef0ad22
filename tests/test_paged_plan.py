"""GPU checks of fa_cache_plan where a batch holds something that does not fit
or has no room: that request keeps what it has, and the others are served."""

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

from io_aware_exact_tiled_gb300 import binding as fb
from io_aware_exact_tiled_gb300 import build as fbuild
from oracle import paged as P
from test_paged import PLAN_KEYS, make_plan, run_plan

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def refuse(x, b):
    """The lists that a plan of x leaves when it refuses request b: those of a
    plan in which b brings nothing, with -1 for the slots of b's tokens."""
    y = {k: np.array(v) if isinstance(v, np.ndarray) else v for k, v in x.items()}
    n = max(int(x["new_len"][b]), 0)
    y["new_len"][b] = y["cache_len"][b] = 0
    want = P.plan(**{**y, "total": x["total"] - n})
    at = want["cu_seqlens"][b]
    want["slots"] = np.insert(want["slots"], at, np.full(n, -1))
    want["cu_seqlens"][b + 1:] += n
    want["cache_len"][b] = x["cache_len"][b]
    return want


@pytest.mark.parametrize("B", [6, 1500])
@pytest.mark.parametrize("n", [-1, 0, 9])
@pytest.mark.parametrize("length", [-1, -5, -(1 << 31), "above", (1 << 31) - 1])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_cached_length_out_of_range_is_refused(cuda_device, B, n, length, in_place):
    """Released ones too: no block of theirs goes back, none is handed out."""
    x = make_plan(B, 16, 60, 20, 0.2, 1.0, seed=B + 7)
    b = B // 2
    had = -(-int(x["cache_len"][b]) // 16)
    x["total"] += n - max(int(x["new_len"][b]), 0) if n > 0 else 0
    x["new_len"][b] = n
    x["cache_len"][b] = 16 * x["block_table"].shape[1] + 1 if length == "above" else length
    # (the ring has room for every block that it could get)
    assert had <= x["block_table"].shape[1]
    want = refuse(x, b)
    got, status = run_plan(x, cuda_device, in_place)
    for k in PLAN_KEYS:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    assert status == fb.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("n", [200, 1 << 30, (1 << 31) - 1])
def test_a_new_length_above_the_table_is_refused(cuda_device, n):
    """It also takes every later request past total, so these are refused too:
    none of them may change."""
    x = make_plan(8, 16, 60, 20, 0.0, 1.0, seed=3)
    b = 5
    x["new_len"][b] = n
    got, status = run_plan(x, cuda_device)
    assert status == fb.FA_ERR_INVALID_ARG
    np.testing.assert_array_equal(got["cache_len"][b:], x["cache_len"][b:])
    np.testing.assert_array_equal(got["block_table"][b:], x["block_table"][b:])
    front = P.plan(**{**x, "new_len": np.where(np.arange(8) < b, x["new_len"], 0)})
    for k in ("cache_len", "block_table"):
        np.testing.assert_array_equal(got[k][:b], front[k][:b])
    np.testing.assert_array_equal(got["free_state"], front["free_state"])
    t0 = front["cu_seqlens"][b]
    np.testing.assert_array_equal(got["slots"][:t0], front["slots"][:t0])
    assert (got["slots"][t0:] == -1).all()


def test_entries_that_are_no_blocks_get_no_slots(cuda_device):
    """Tokens in front of and behind a bad table or ring entry keep their slots;
    a bad ring entry is carried into the table, where attention reports it."""
    x = make_plan(4, 16, 60, 0, 0.0, 1.0, seed=2)
    x["cache_len"][:] = [20, 30, 0, 40]
    nb = 40
    table = np.full((4, 6), -1)
    table[0, :2], table[1, :2], table[3, :3] = [3, 4], [5, 6], [7, 8, 9]
    ring = np.full(nb, -1)
    ring[:8] = [10, 1 << 20, 12, 13, -7, 15, 16, 17]
    x.update(block_table=table, free_blocks=ring, free_state=np.array([0, 8]), new_len=np.array([30, 1, 40, 2]),
             total=73)
    x["block_table"][1, 1] = nb            # request 1's last block
    got, status = run_plan(x, cuda_device)
    assert status == fb.FA_ERR_INVALID_ARG
    want = P.plan(**x)                     # the lists as if every entry were a block
    for k in ("cache_len", "block_table", "free_blocks", "free_state", "cu_seqlens"):
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    bad = (want["slots"] < 0) | (want["slots"] >= nb * 16)
    assert 0 < bad.sum() < 73
    np.testing.assert_array_equal(got["slots"], np.where(bad, -1, want["slots"]))


@pytest.mark.parametrize("B,bs,len_hi,new_hi,release,room", [
    (1025, 64, 500, 9, 0.1, 0.9), (5000, 16, 64, 40, 0.2, 0.6), (16384, 16, 20, 2, 0.1, 0.99),
    (2, 64, 70, 40000, 0.0, 1.0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_large_plans_in_a_smaller_cluster(cuda_device, B, bs, len_hi, new_hi, release, room, in_place, monkeypatch):
    """Where the device cannot hold a cluster of sixteen CTAs (here: a build
    that asks for two at most) a large plan is the same."""
    dbg, regular = ctypes.CDLL(fbuild.build_debug()), fb.load()
    for name in ("fa_cache_plan", "fa_get_status"):
        getattr(dbg, name).argtypes = getattr(regular, name).argtypes
        getattr(dbg, name).restype = getattr(regular, name).restype
    x = make_plan(B, bs, len_hi, new_hi, release, room, seed=B + bs)
    want = P.plan(**x)
    monkeypatch.setattr(fb, "_lib", dbg)
    got, status = run_plan(x, cuda_device, in_place)
    for k in PLAN_KEYS:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    assert status == (fb.FA_ERR_NO_BLOCKS if want["refused"] else fb.FA_OK)


def test_a_large_plan_is_captured_as_a_process_first_call(cuda_device):
    """What the first large plan asks the device is allowed under capture."""
    code = """
import torch, io_aware_exact_tiled_gb300 as fa
c = fa.paged_cache(9000, 1, 16, 64, 4500, 2)
new = torch.ones(4500, dtype=torch.int32, device="cuda")
cu, slots = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (4501, 4500))
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    fa.cache_plan(new, c.cache_len, c.block_table, c.free_blocks, c.free_state, 16, cu_seqlens=cu, slots=slots,
                  ws=c.status)
for _ in range(17):
    g.replay()
assert fa.get_status(c.status) == 0 and (c.cache_len == 17).all() and c.free_state.tolist() == [0, 0]
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
