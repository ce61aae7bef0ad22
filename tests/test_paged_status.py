"""Whether a plan found its blocks can be read through the cache's own status
buffer, as the documented serving step does."""

import os

import pytest
import torch

import io_aware_exact_tiled_gb300 as fa
from io_aware_exact_tiled_gb300 import binding as fb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def readme_step():
    text = open(os.path.join(ROOT, "README.md")).read()
    start = text.index("```python", text.index("A serving step over the paged cache")) + len("```python")
    return text[start:text.index("```", start)]


def test_a_cache_comes_with_a_status_buffer():
    c = fa.paged_cache(4, 1, 16, 64, 2, 4, device="cpu")
    assert c.status.dtype == torch.uint8 and c.status.numel() == 256 and not c.status.any()
    assert len(c) == 8 and c._fields[-1] == "free_state" and fa.PagedCache(*c).status is None
    assert "ws=c.status" in readme_step() and "get_status(c.status)" in readme_step()


@pytest.mark.gpu
def test_a_refusal_is_seen(cuda_device):
    c = fa.paged_cache(3, 1, 16, 64, 2, 4, cuda_device)
    new = torch.tensor([30, 30], dtype=torch.int32, device=cuda_device)
    args = (new, c.cache_len, c.block_table, c.free_blocks, c.free_state, 16)
    cu, slots = fa.cache_plan(*args, total=60, ws=c.status)
    assert fa.get_status(c.status) == fb.FA_ERR_NO_BLOCKS
    assert (slots[:30] >= 0).all() and (slots[30:] == -1).all() and c.cache_len.tolist() == [30, 0]
    new.copy_(torch.tensor([-1, 30]))
    fa.cache_plan(*args, total=60, ws=c.status)          # its blocks come back: from the next plan on
    assert fa.get_status(c.status) == fb.FA_ERR_NO_BLOCKS
    new[0] = 0
    fa.cache_plan(*args, total=60, ws=c.status)
    assert fa.get_status(c.status) == fb.FA_OK and c.cache_len.tolist() == [0, 30]


@pytest.mark.gpu
def test_the_documented_step_runs(cuda_device):
    """The README's step, on a smaller cache, for a prompt and for one that
    finds no blocks."""
    code = readme_step().replace("4096", "6").replace("B=64, max_blocks=256", "B=2, max_blocks=8")
    make, step = code.strip().split("\n", 1)
    step = step.replace("max_new=1", "max_new=int(new_len.max())")
    env = {"fa": fa}
    exec(make, env)
    for new, refused in (([100, 64], 0), ([1, 300], 300)):
        total = sum(new)
        env["new_len"] = torch.tensor(new, dtype=torch.int32, device=cuda_device)
        env["q"] = torch.randn((total, 32, 128), device=cuda_device).to(torch.bfloat16)
        env["k"], env["v"] = (torch.randn((total, 8, 128), device=cuda_device).to(torch.bfloat16) for _ in range(2))
        env["retry"] = ()
        exec(step, env)
        assert len(env["retry"]) == refused and env["o"].shape == env["q"].shape
        assert torch.isfinite(env["o"]).all()
