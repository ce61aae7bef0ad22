"""Give-up of the paged row-tile kernel: a debug build (0.2 s limit) withholds
one "P ready" arrival of each row tile's first softmax warp, so the product
issuers' waits run out. Every role has to leave, the call reports
FA_ERR_TIMEOUT, and the context stays usable. Nothing faults or hangs."""

import ctypes

import pytest
import torch

import io_aware_exact_tiled_gb300 as fa
from io_aware_exact_tiled_gb300 import binding as fb
from io_aware_exact_tiled_gb300 import build as fbuild

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,n", [(64, 300), (128, 40)])
def test_row_tile_kernel_reports_timeout(cuda_device, d, n, monkeypatch):
    Hkv, G, bs = 2, 2, 64
    c = fa.paged_cache(40, Hkv, bs, d, 2, 16, cuda_device)
    gen = torch.Generator(device=cuda_device).manual_seed(0)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device=cuda_device).to(torch.bfloat16)

    new = torch.tensor([n, 70], dtype=torch.int32, device=cuda_device)
    total = n + 70
    cu, slots = fa.cache_plan(new, c.cache_len, c.block_table, c.free_blocks, c.free_state, bs, total=total)
    fa.cache_append(rand(total, Hkv, d), rand(total, Hkv, d), c.k, c.v, c.k_scale, c.v_scale, slots)
    q = rand(total, Hkv * G, d)
    args = (q, c.k, c.v, c.k_scale, c.v_scale, cu, c.cache_len, c.block_table, max(n, 70))
    want = fa.forward_paged(*args)
    torch.cuda.synchronize()

    dbg = ctypes.CDLL(fbuild.build_debug())
    regular = fb.load()
    for name in ("fa_fwd_paged", "fa_fwd_paged_workspace_size", "fa_get_status"):
        getattr(dbg, name).argtypes = getattr(regular, name).argtypes
        getattr(dbg, name).restype = getattr(regular, name).restype
    ws = fa.workspace(fa.fwd_paged_workspace_size(2, Hkv * G, Hkv, total, max(n, 70), d), cuda_device)
    monkeypatch.setattr(fb, "_lib", dbg)
    fa.forward_paged(*args, ws=ws)
    assert fa.get_status(ws) == fb.FA_ERR_TIMEOUT
    assert fa.get_status(ws) == fb.FA_OK                 # reading clears the word
    monkeypatch.setattr(fb, "_lib", regular)

    o, lse = fa.forward_paged(*args, ws=ws)
    assert fa.get_status(ws) == fb.FA_OK
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
