"""Limits of the cache in pages that are refused before anything is launched (no GPU)."""
import pytest

import exact_top_token_gb300 as hk
from test_pages_host import OK, SMALL, UNSUPPORTED, calls_of


@pytest.fixture(scope="module")
def lib():
    hk.build()
    return hk.load()


@pytest.mark.parametrize("name", ["fork", "free", "grow", "compact"])
def test_pages_of_a_pool(lib, name):
    """Page numbers a few thousand past the pool's end have to fit 32 bits."""
    call = calls_of(lib)[name]
    for N in ((1 << 30) + 1, (1 << 31) - 4096, (1 << 31) - 1):
        assert call(N=N) == UNSUPPORTED, N
        assert lib.hytopk_page_workspace_size(N) == 0
    most = 1 << 30
    need = lib.hytopk_page_workspace_size(most)
    assert need >= 8 * most
    if name in ("fork", "free"):
        assert call(N=most, count=0) == OK
    else:
        assert call(N=most, wb=need - 1) == SMALL
