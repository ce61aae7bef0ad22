"""fa_cache_plan's workspace argument, and what the library refuses on the
host before any launch."""

import pytest

from io_aware_exact_tiled_gb300 import binding as fb
from io_aware_exact_tiled_gb300 import build as fbuild

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fb.load()


@pytest.mark.parametrize("ws,size", [(None, 256), (FAKE + 16, 256), (FAKE + 128, 256), (FAKE, 0), (FAKE, 255)])
def test_plan_refuses_a_workspace_that_is_none(lib, ws, size):
    assert lib.fa_cache_plan(*[FAKE] * 9, 4, 8, 64, 16, 4, ws, size, None) == fb.FA_ERR_INVALID_ARG


def test_plan_without_tokens_needs_no_slots(lib):
    """slots may be null when total is 0: then only the workspace is wrong."""
    p = [FAKE] * 8 + [None]
    assert lib.fa_cache_plan(*p, 4, 8, 64, 16, 1, FAKE, 256, None) == fb.FA_ERR_INVALID_ARG
    assert lib.fa_cache_plan(*p, 4, 8, 64, 16, 0, FAKE, 128, None) == fb.FA_ERR_INVALID_ARG
