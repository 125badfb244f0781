"""Page-management calls report tables and counts that do not fit, as the oracle does."""
import pytest
import torch

from sparse_long_context_min_b200 import binding as B
from test_gpu_pages import Both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [6, 1200])   # released and counted in one launch, and in two
def test_fork_of_a_last_page_beyond_the_pool(rows):
    s = Both(40, rows, 30)
    lens = [50, 33, 16] + [0] * (rows - 3)
    s.reserve(lens)
    s.set_lens(lens)
    s.table[1, 2] = s.o.table[1][2] = 40      # the page that row 1 ends inside of
    more = list(range(100, rows))             # (pairs without tokens)
    s.fork([1] + [3] * len(more), [4] + more)
    s.fork([1, 0] + [3] * len(more), [4, 5] + more)
    assert s.o.lens[4] == 33 and s.o.table[4][2] == -1 and s.o.lens[5] == 50


@pytest.mark.parametrize("page", [1, 37])
def test_compact_with_an_entry_of_a_free_page(page):
    """A table names a page whose count is zero: below the pages in use, where another page moves to, and above."""
    s = Both(40, 3, 20)
    s.reserve([300, 260, 0])
    s.set_lens([300, 260, 0])
    s.free([0])
    s.reserve([40, 260, 20])
    s.set_lens([40, 260, 20])
    assert s.o.ref[page] == (page == 1)
    if page == 1:
        s.ref[1] = s.o.ref[1] = 0             # row 0's second page
        assert s.o.table[0][1] == 1
    else:
        s.table[0, 1] = s.o.table[0][1] = page
        s.ref[1] = s.o.ref[1] = 0
    s.compact()
    s.free(None)
