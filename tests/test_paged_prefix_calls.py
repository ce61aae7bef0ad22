"""GPU checks of attention over shared prefixes as calls: how many kernels each
way of joining runs, and calls that run at the same time."""

import pytest
import torch

import io_aware_exact_tiled_gb300 as fa

from test_paged_prefix import Batch

pytestmark = pytest.mark.gpu

WAYS = {
    # requests, groups, key heads, heads of a group, d, kernels
    "split keys in both passes": ([(5, 1)] * 3, [(0, 200)], 1, 4, 64, 2),
    "one row tile beside split keys": ([(5, 1)] * 30, [(0, 900)], 2, 4, 128, 3),
    "two row tiles beside split keys": ([(5, 1)] * 80, [(0, 900)], 2, 4, 64, 3),
    "prompts": ([(0, 130), (10, 40)], [(0, 900)], 2, 2, 64, 3),
    "prompts, one row tile": ([(0, 40)] * 4, [(i, 300) for i in range(4)], 2, 2, 128, 4),
    "long prompts": ([(0, 300)] * 5, [(0, 300), (2, 5000)], 4, 4, 128, 3),
}


@pytest.mark.parametrize("way", list(WAYS))
def test_kernels_of_each_way_of_joining(cuda_device, way):
    pairs, groups, Hkv, G, d, kernels = WAYS[way]
    b = Batch(pairs, groups, 32, Hkv, G, d, cuda_device)
    b.check()
    assert fa.last_launch_count() == kernels


def test_calls_at_the_same_time(cuda_device):
    """Calls of every way on streams of their own, each with its workspace."""
    batches = [Batch(*WAYS[w][:2], 32, *WAYS[w][2:5], cuda_device, seed=i) for i, w in enumerate(WAYS)]
    want = [b.run() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    args, outs, spaces = [b.tensors() for b in batches], [], []
    for b in batches:
        Hq, n = b.Hkv * b.G, b.q.shape[0]
        outs.append((torch.full_like(b.q, 7.0), torch.full((Hq, n), 7.0, device=cuda_device)))
        spaces.append(fa.workspace(fa.fwd_paged_prefix_workspace_size(len(b.lens), len(b.plen), Hq, b.Hkv, n,
                                                                      max(b.new), b.d), cuda_device).fill_(255))
    torch.cuda.synchronize()
    for _ in range(20):
        for b, a, (o, lse), ws, s in zip(batches, args, outs, spaces, streams):
            fa.forward_paged_prefix(b.q, *a, max(b.new), scale=b.scale, out=o, lse=lse, ws=ws, stream=s)
    torch.cuda.synchronize()
    for w, g in zip(want, outs):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])
