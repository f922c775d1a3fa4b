"""What kvsel_attend_tree promises whichever way the work is cut."""
import numpy as np
import pytest

from tests import cache_harness as CH
from tests import step_harness as SH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    yield


@pytest.mark.parametrize("B,m,G", [(304, 8, 4), (304, 24, 8)])
def test_items_that_nobody_joins_leave_no_records(B, m, G):
    # two whole items per SM (152 of them): a record for each would lie behind the room that records have
    c = SH.TreeCase(B=B, H=1, G=G, m=m, lens=[m + i % 50 for i in range(B)], layout="contiguous", seed=m).upload()
    ws = c.call()
    assert CH.status(ws) == 0
    assert bool((ws[256 + 65536:] == 0xFF).all())
    c.check()


@pytest.mark.parametrize("B,H,m,G,bound", [(48, 8, 1, 4, 8192), (48, 8, 4, 4, 8192), (12, 8, 4, 4, 131072), (1, 8, 16, 1, 300),
                                           (64, 4, 2, 8, 4096), (200, 1, 3, 5, 1000), (3, 2, 1, 16, 20000), (304, 1, 16, 1, 256)])
def test_weights_of_few_rows_are_kept_whatever_the_bound(B, H, m, G, bound):
    # short texts under a large max_len, many segments and few: up to 16 query rows under the bound of the kernel of few rows
    lens = [[m + 7 * (i + 3 * h) % 120 for h in range(H)] for i in range(B)]
    c = CH.paired(SH.TreeCase(B=B, H=H, G=G, m=m, lens=lens, layout="packed", logit=0.1, pad_rows=bound - max(map(max, lens)), seed=B + m)).upload()
    assert CH.status(c.call()) == 0
    c.check()
    CH.check_tokens(c)


@pytest.mark.parametrize("m,G", [(1, 4), (4, 4), (3, 5), (16, 1)])
@pytest.mark.parametrize("layout,block", [("contiguous", 0), ("paged", 16)])
@pytest.mark.parametrize("n,pad", [(700, 0), (5000, 0), (300, 9000)])
def test_weights_of_few_rows_over_longer_texts(m, G, layout, block, n, pad):
    c = CH.paired(SH.TreeCase(B=2, H=2, G=G, m=m, lens=[n, 90], layout=layout, block=block, logit=0.1, pad_rows=pad, seed=n + m)).upload()
    assert CH.status(c.call()) == 0
    c.check()
    CH.check_tokens(c)
