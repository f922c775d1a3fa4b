"""Numbers on the device that lie far out of range: offsets of a packed cache near the ends of 64 bits."""
import numpy as np
import pytest

from tests import cache_harness as CH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    from kv_cache_eviction_window_gb300 import binding

    binding.load()
    yield


@pytest.mark.parametrize("m", [1, 6, 40])
@pytest.mark.parametrize("acc", [False, True])
def test_offsets_anywhere_in_64_bits(m, acc):
    # rows of a segment outside the packed cache: it counts as empty, the other keeps its result
    n = 200
    c = CH.Case(lens=n, m=m, layout="packed", seed=m).upload()
    ora = c.oracle()
    ora[0][1] = {x: np.full_like(y, -np.inf if x == "lse" else 0.0) for x, y in ora[0][1].items()}
    for first in (2 ** 63 - 1, 2 ** 63 - n, 2 ** 63 - n + 1, 2 ** 62, 2 ** 32, n + 1, -1, -n, -2 ** 63, -2 ** 63 + n):
        c.offsets[1] = first
        c.t["acc"].zero_()
        ws = c.call(acc=acc)
        assert CH.status(ws) == -7, first
        c.check(ora, acc=acc)
