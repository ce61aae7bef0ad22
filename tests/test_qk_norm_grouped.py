"""GPU checks of the norm's gradient where keys have fewer heads than queries
and a warp takes several tokens: every row of a gradient is its own token's."""

import pytest
import torch

import io_aware_exact_tiled_gb300 as fa

from test_qk_norm import Case

pytestmark = pytest.mark.gpu

HEADS = [(128, 32, 8), (128, 28, 4), (128, 64, 8), (128, 16, 2), (64, 64, 8), (64, 24, 6), (64, 5, 40)]


def gradients(c):
    x, up = c.split(c.qkv), c.split(c.up)
    return fa.qk_norm_rope_backward(x["q"], x["k"], up["q"], up["k"], **c.kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,Hq,Hkv", HEADS)
@pytest.mark.parametrize("tokens", [200, 350, 500, 1000, 1100, 1215])
def test_gradient_of_grouped_heads(cuda_device, tokens, d, Hq, Hkv, dtype):
    """Token counts on both sides of what one pass over the GPU's warps takes,
    packed and (every other one) dense, whose two rows are the tokens' halves."""
    if (tokens + Hq) % 4:
        c = Case(cuda_device, "packed", d, d, Hq, Hkv, False, "qk", dtype, lens=(tokens // 3, 0, 1, tokens - tokens // 3 - 1))
    else:
        c = Case(cuda_device, "dense", d, d // 2, Hq, Hkv, True, "qk", dtype, lens=(tokens // 2,))
    a = gradients(c)
    c.check_backward({"q": a[0], "k": a[1]}, {"q": a[2], "k": a[3]})


@pytest.mark.parametrize("norms", ["", "q", "k"])
def test_gradient_of_grouped_heads_without_a_weight(cuda_device, norms):
    for d, Hq, Hkv in HEADS[:2]:
        c = Case(cuda_device, "packed", d, d, Hq, Hkv, False, norms, torch.bfloat16, lens=(700, 300))
        a = gradients(c)
        c.check_backward({"q": a[0], "k": a[1]}, {"q": a[2], "k": a[3]})
