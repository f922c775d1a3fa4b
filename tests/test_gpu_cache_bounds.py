"""Numbers on the device that lie far out of range: offsets of a packed cache near the ends of 64 bits,
and what a workspace may hold where a call that gave up has written no records."""
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


@pytest.mark.parametrize("B,H,m,G", [(2, 2, 6, 7), (2, 2, 16, 4)])
def test_a_join_follows_no_stray_record(B, H, m, G):
    """A call that gives up on a wait may leave records of its items unwritten; the join then finds what
    the workspace held before, here records whose sum passes 32 bits."""
    import torch

    from kv_cache_eviction_window_gb300 import binding as L

    c = CH.Case(B=B, G=G, H=H, m=m, lens=[2000, 900], layout="paged", seed=m).upload()
    good = dict(c.params)
    ws = CH.workspace(L.kvsel_attend_workspace_size(L.make_attn_params(**good), False))
    records = ws[256 + 65536:256 + 65536 + 8 * B * H].view(torch.int32).view(-1, 2)
    c.params["wait_cycles"] = 1
    for first, follow in ((151, 2 ** 31 - 101), (1, 2 ** 31 - 1), (0, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1), (152, 0), (140, 12)):
        records[:, 0], records[:, 1] = first, follow
        c.call(ws=ws)
        assert CH.status(ws) == -6
    c.params = good
    c.t["out"].fill_(7.0)
    c.t["lse"].fill_(7.0)
    c.call(ws=ws)
    assert CH.status(ws) == 0
    c.check()
