"""Give-up of the paged split-key kernel: a debug build (0.2 s limit) does not
request the first chunk's V in one warp of each CTA, so that this warp's wait
runs out, in a long piece (whose other warps wait at its barrier) or in a short
unit of its own. Every warp has to leave, the call reports FA_ERR_TIMEOUT, and
the context stays usable. Nothing faults or hangs."""

import ctypes

import pytest
import torch

import io_aware_exact_tiled_gb300 as fa
from io_aware_exact_tiled_gb300 import binding as fb
from io_aware_exact_tiled_gb300 import build as fbuild

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,bs,B,length", [(64, 64, 1, 9000), (128, 16, 2, 3000), (64, 16, 400, 40),
                                           (128, 64, 400, 70)])
def test_split_key_kernel_reports_timeout(cuda_device, d, bs, B, length, monkeypatch):
    Hkv, G = 2, 4
    blocks = -(-length // bs)
    c = fa.paged_cache(B * blocks, Hkv, bs, d, B, blocks, cuda_device)
    gen = torch.Generator(device=cuda_device).manual_seed(0)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device=cuda_device).to(torch.bfloat16)

    new = torch.full((B,), length, dtype=torch.int32, device=cuda_device)
    _, slots = fa.cache_plan(new, c.cache_len, c.block_table, c.free_blocks, c.free_state, bs, total=B * length)
    fa.cache_append(rand(B * length, Hkv, d), rand(B * length, Hkv, d), c.k, c.v, c.k_scale, c.v_scale, slots)
    cu = torch.arange(B + 1, dtype=torch.int32, device=cuda_device)
    q = rand(B, Hkv * G, d)
    args = (q, c.k, c.v, c.k_scale, c.v_scale, cu, c.cache_len, c.block_table, 1)
    want = fa.forward_paged(*args)
    torch.cuda.synchronize()

    dbg = ctypes.CDLL(fbuild.build_debug())
    regular = fb.load()
    for name in ("fa_fwd_paged", "fa_fwd_paged_workspace_size", "fa_get_status"):
        getattr(dbg, name).argtypes = getattr(regular, name).argtypes
        getattr(dbg, name).restype = getattr(regular, name).restype
    ws = fa.workspace(fa.fwd_paged_workspace_size(B, Hkv * G, Hkv, B, 1, d), cuda_device)
    monkeypatch.setattr(fb, "_lib", dbg)
    fa.forward_paged(*args, ws=ws)
    assert fa.get_status(ws) == fb.FA_ERR_TIMEOUT
    assert fa.get_status(ws) == fb.FA_OK                 # reading clears the word
    monkeypatch.setattr(fb, "_lib", regular)

    o, lse = fa.forward_paged(*args, ws=ws)
    assert fa.get_status(ws) == fb.FA_OK
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
