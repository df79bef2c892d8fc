"""The pool of a cache in pages (GPU) at the edges of what its entry points take, against
tests/pages_oracle.py."""
import pytest

import exact_top_token_gb300 as hk
from test_gpu_pages_pool import Both

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    hk.build()


@pytest.mark.parametrize("wanted", [10, 11, 12, 500])
def test_nothing_is_granted_behind_what_an_empty_pool_lacks(wanted):
    """All pages are free, and the first sequence wants as many or more; those behind it want
    none (their last page is not there), or some."""
    t = Both(4, 600, 10, 16, [0, 5, 0, 0])
    t.refs[t.table[1, 0]] = t.o.refs[t.o.table[1][0]] = 0
    t.table[1, 0] = t.o.table[1][0] = -1
    t.grow([16 * wanted, 1, 0, 1])
    assert t.word.item() == hk.DEV_NO_PAGE
    assert t.lengths.tolist() == ([160, 6, 0, 0] if wanted == 10 else [0, 5, 0, 0])


@pytest.mark.parametrize("N", [1, 40, 5000])
def test_a_pool_that_no_sequence_uses(N):
    """A table without rows: pages are counted all the same."""
    t = Both(0, 3, N, 16, [])
    t.refs[N // 2] = t.o.refs[N // 2] = 1
    t.compact()
    t.grow([])
    t.free([])
    t.fork([], [])
