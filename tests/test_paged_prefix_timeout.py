"""Give-up of attention with shared prefixes: a debug build (0.2 s limit)
withholds a "P ready" arrival of each row tile and a copy of each split-key
CTA, so waits run out in both passes. Every kernel of the chain has to end, the
call reports FA_ERR_TIMEOUT, and the context stays usable. Nothing faults or
hangs."""

import ctypes

import pytest
import torch

import io_aware_exact_tiled_gb300 as fa
from io_aware_exact_tiled_gb300 import binding as fb
from io_aware_exact_tiled_gb300 import build as fbuild

from test_paged_prefix import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs,prefix,G,d", [
    ([(40, 1), (700, 1)], 900, 4, 128),                # split keys in both passes
    ([(60, 1)] * 12, 5000, 4, 64),                     # one row tile, 48 rows, beside split keys
    ([(60, 1)] * 30, 3000, 4, 128),                    # one row tile, 120 rows
    ([(60, 1)] * 80, 3000, 4, 128),                    # two row tiles
    ([(0, 300), (10, 40)], 1000, 2, 64)])              # prompts: row tiles in both
def test_chain_reports_timeout(cuda_device, monkeypatch, pairs, prefix, G, d):
    b = Batch(pairs, [(0, prefix)], 64, 2, G, d, cuda_device)
    want = b.run()
    dbg = ctypes.CDLL(fbuild.build_debug())
    regular = fb.load()
    for name in ("fa_fwd_paged_prefix", "fa_fwd_paged_prefix_workspace_size", "fa_get_status"):
        getattr(dbg, name).argtypes = getattr(regular, name).argtypes
        getattr(dbg, name).restype = getattr(regular, name).restype
    monkeypatch.setattr(fb, "_lib", dbg)
    b.run(status=fb.FA_ERR_TIMEOUT)
    monkeypatch.setattr(fb, "_lib", regular)
    got = b.run()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
