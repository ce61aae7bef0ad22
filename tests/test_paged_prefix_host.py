"""Workspace of attention over shared prefixes on the CPU: what a call does not
use it does not ask for."""

import pytest

from io_aware_exact_tiled_gb300 import binding as fb
from io_aware_exact_tiled_gb300 import build as fbuild


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fb.load()


@pytest.mark.parametrize("d", [64, 128])
def test_rows_are_kept_once_for_each_pass_that_leaves_them(lib, d):
    """Output in fp32, maximum and sum of each row: the prefixes' pass's, and the
    own pass's too where both run at once (decoding), but not with prompts."""
    Hq, Hkv, B, P = 32, 8, 64, 4

    def growth(max_new):
        a, b = (lib.fa_fwd_paged_prefix_workspace_size(B, P, Hq, Hkv, n, max_new, d) for n in (20000, 40000))
        return b - a

    rows = 20000 * Hq * (d + 2) * 4
    few = 1 << 20                                        # counters of the row tiles
    assert 2 * rows <= growth(1) <= 2 * rows + few
    assert rows <= growth(5000) <= rows + few
