"""GPU check of the norm's angles at the farthest positions."""

import numpy as np
import pytest
import torch

import io_aware_exact_tiled_gb300 as fa
from oracle import qk_norm as N

pytestmark = pytest.mark.gpu

# The angle is within 2^-33 of a turn, its fraction then rounded to 2^-32 (half of that off): 2^-32 of a
# turn, 1.5e-9 radians. What is left of a quarter turn (at most pi / 4) is rounded to fp32 and multiplied
# (half a step each: 2^-25 each below 1, times the slope of at most 1), the series' last product and sum
# round once each (2^-25), its other terms' roundings are below 2^-26 together, as is what it leaves out.
# A row (1, 0) without a norm becomes (cos, sin) with no further rounding.
TOLERANCE = 5 * 2.0 ** -25


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("last", [2 ** 31 - 1, 2 ** 30 + 12345, -(2 ** 31) + 100])
def test_angles_of_far_positions(cuda_device, last, sign, inter):
    """Frequencies of either sign, of whole turns a position and of tiny parts
    of one, at positions near the ends of 32 bits."""
    d, n = 128, 64
    rng = np.random.default_rng(5)
    f = sign * np.concatenate([1e4 ** (-np.arange(0, 64, 2) / 64), [0.3, 1.7, 1e6 + 0.3, 1e11 / 3, 6.283185307179586],
                               2.0 ** -rng.uniform(1, 45, 27)])
    x = torch.zeros(1, 1, n, d, device=cuda_device)
    u, v = (np.arange(0, d, 2), np.arange(1, d, 2)) if inter else (np.arange(d // 2), np.arange(d // 2) + d // 2)
    x[..., u] = 1.0
    z, _ = fa.qk_norm_rope(x, x, torch.tensor(f, device=cuda_device), interleaved=inter,
                           ends=torch.tensor([last], dtype=torch.int32, device=cuda_device))
    a = N.angles(last - n + np.arange(n), f)
    z = z[0, 0].double().cpu().numpy()
    assert np.abs(z[:, u] - np.cos(a)).max() <= TOLERANCE
    assert np.abs(z[:, v] - np.sin(a)).max() <= TOLERANCE
