"""Tokens taken back between plans (rejected drafts): lengths are lowered, and
blocks that the shorter length does not reach go to the back of the ring. No
block is lost or handed out twice, with the definition and with the kernel."""

import numpy as np
import pytest
import torch

import io_aware_exact_tiled_gb300 as fa
from io_aware_exact_tiled_gb300 import binding as fb
from oracle import paged as P

BS, NB, MB, B = 16, 40, 8, 4


def take_back(x, b, new):
    """Lowers request b's length by the documented rule."""
    had, keep = -(-int(x["cache_len"][b]) // BS), -(-new // BS)
    head, count = (int(v) for v in x["free_state"])
    for j in range(keep, had):
        x["free_blocks"][(head + count) % NB] = x["block_table"][b, j]
        count += 1
    x["free_state"][1] = count
    x["cache_len"][b] = new


def owned(x):
    """Blocks of the tables and of the ring."""
    mine = [x["block_table"][b, j] for b in range(B) for j in range(-(-int(x["cache_len"][b]) // BS))]
    head, count = (int(v) for v in x["free_state"])
    return mine + [x["free_blocks"][(head + i) % NB] for i in range(count)]


def serve(plan_once, seed):
    rng = np.random.default_rng(seed)
    x = dict(cache_len=np.zeros(B, np.int32), block_table=np.full((B, MB), -1, np.int32),
             free_blocks=np.arange(NB, dtype=np.int32), free_state=np.array([0, NB], np.int32))
    fell = 0
    for _ in range(60):
        new = rng.integers(0, 20, B)
        new[rng.random(B) < 0.1] = -1
        new = np.where(x["cache_len"] + new > MB * BS, -1, new)
        x = plan_once(x, new)
        assert sorted(owned(x)) == list(range(NB))
        for b in range(B):
            back = int(rng.integers(0, min(20, int(x["cache_len"][b])) + 1))
            fell += -(-int(x["cache_len"][b]) // BS) - -(-(int(x["cache_len"][b]) - back) // BS)
            take_back(x, b, int(x["cache_len"][b]) - back)
        assert sorted(owned(x)) == list(range(NB))
    assert fell > 20


@pytest.mark.parametrize("seed", range(5))
def test_no_block_is_lost_by_the_definition(seed):
    def once(x, new):
        r = P.plan(new, x["cache_len"], x["block_table"], x["free_blocks"], x["free_state"], BS,
                   int(new.clip(0).sum()))
        assert not r["refused"]
        return {k: r[k] for k in x}

    serve(once, seed)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(3))
def test_no_block_is_lost_by_the_kernel(cuda_device, seed):
    c = fa.paged_cache(NB, 1, BS, 64, B, MB, cuda_device)
    names = ("cache_len", "block_table", "free_blocks", "free_state")

    def once(x, new):
        for k in names:
            getattr(c, k).copy_(torch.from_numpy(x[k]))
        total = int(new.clip(0).sum())
        n = torch.tensor(new, dtype=torch.int32, device=cuda_device)
        _, slots = fa.cache_plan(n, c.cache_len, c.block_table, c.free_blocks, c.free_state, BS, total=total,
                                 ws=c.status)
        assert fa.get_status(c.status) == fb.FA_OK and (slots >= 0).all()
        return {k: getattr(c, k).cpu().numpy() for k in names}

    serve(once, seed)


@pytest.mark.gpu
@pytest.mark.parametrize("back", [1, 3, 15, 16, 17, 30])
def test_attention_after_tokens_were_taken_back(cuda_device, back):
    """The cache then holds what it would have held without the rejected tokens
    (their scale is no larger here)."""
    gen = torch.Generator(device=cuda_device).manual_seed(back)
    kv = torch.randn((2, 80, 1, 64), generator=gen, device=cuda_device).to(torch.bfloat16)
    kv[:, :, :, 0] = 4.0                                   # every block's largest value
    q = torch.randn((80, 2, 64), generator=gen, device=cuda_device).to(torch.bfloat16)
    twins = [fa.paged_cache(NB, 1, BS, 64, 1, MB, cuda_device) for _ in range(2)]

    def step(c, rows):
        n = torch.tensor([len(rows)], dtype=torch.int32, device=cuda_device)
        cu, slots = fa.cache_plan(n, c.cache_len, c.block_table, c.free_blocks, c.free_state, BS, total=len(rows),
                                  ws=c.status)
        fa.cache_append(kv[0][rows], kv[1][rows], c.k, c.v, c.k_scale, c.v_scale, slots)
        assert fa.get_status(c.status) == fb.FA_OK
        return fa.forward_paged(q[rows], c.k, c.v, c.k_scale, c.v_scale, cu, c.cache_len, c.block_table, len(rows))

    step(twins[0], list(range(33)))
    step(twins[0], list(range(40, 40 + back)))             # rejected
    x = {k: getattr(twins[0], k).cpu().numpy() for k in ("cache_len", "block_table", "free_blocks", "free_state")}
    take_back(x, 0, 33)
    for k, v in x.items():
        getattr(twins[0], k).copy_(torch.from_numpy(v))
    step(twins[1], list(range(33)))
    a, b = (step(c, list(range(33, 36))) for c in twins)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert twins[0].free_state[1] == twins[1].free_state[1]
