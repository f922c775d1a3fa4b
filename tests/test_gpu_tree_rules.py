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
