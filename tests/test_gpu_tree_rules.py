"""What kvsel_attend_tree promises whichever way the work is cut."""
import numpy as np
import pytest

from oracle import step_oracle as SO
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


class Windowed(SH.TreeCase):
    """The window counts the tree's rows too."""

    def seen(self, b, h):
        return SO.tree_windowed(int(self.lens[b][h]), self.masks[b], self.window, self.n_sink)

    def run(self):
        self.upload()
        self.params["tree_window"] = True
        assert CH.status(self.call()) == 0
        self.check()


@pytest.mark.parametrize("kind", ["chain", "tree"])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (2, 3), (5, 0), (16, 4), (31, 0), (33, 70), (64, 4), (100, 0)])
@pytest.mark.parametrize("m,G", [(4, 4), (16, 1), (8, 4), (40, 4), (70, 3), (130, 4)])
def test_a_window_that_ends_inside_the_tree(kind, window, n_sink, m, G):
    Windowed(B=2, layout="paged", block=8, lens=[700, m + 2], H=2, G=G, m=m, window=window, n_sink=n_sink, kind=kind, seed=m).run()
    Windowed(lens=m, H=1, G=G, m=m, window=window, n_sink=n_sink, kind=kind, seed=m + 1).run()


@pytest.mark.parametrize("layout,block", [("contiguous", 0), ("packed", 0), ("paged", 16), ("paged", 64)])
@pytest.mark.parametrize("m,window,n_sink", [(300, 40, 0), (1024, 512, 4), (257, 1, 1), (1024, 3, 1100)])
def test_long_chains_under_a_window(layout, block, m, window, n_sink):
    Windowed(B=2, lens=[[m + 70], [m]] if layout == "packed" else [m + 70, m], new=[m, m - 5], H=1, G=2, m=m, layout=layout, block=block, window=window, n_sink=n_sink, kind="chain", seed=m).run()


@pytest.mark.parametrize("m", [3, 20, 64, 150])
def test_any_mask_under_a_window(m):
    g = CH.rng(m)
    for density in (0.1, 0.5, 1.0):
        masks = [g.random((m, m)) < density, np.zeros((m, m), bool), np.ones((m, m), bool)]
        Windowed(B=3, lens=[m + 40, 90 + m, m + 1], m=m, G=4, window=7, n_sink=3, masks=masks, layout="paged", seed=m).run()
    # fewer rows than nodes
    masks = [np.tril(np.ones((m, m), bool))]
    c = Windowed(lens=m - 1, m=m, G=4, masks=masks, window=2, n_sink=1)
    c.seen = lambda b, h: np.array([[masks[0][t, u] and (u > t - 2 or u - 1 < 1) for u in range(1, m)] for t in range(m)])
    c.seen_rows = lambda b, h: np.ones(m - 1, bool)
    c.run()


@pytest.mark.parametrize("m,G,window,n_sink", [(8, 2, 4, 0), (24, 4, 7, 2), (100, 4, 30, 4), (600, 2, 512, 4)])
def test_a_chain_under_a_window_is_causal(m, G, window, n_sink):
    kw = dict(B=2, H=2, G=G, m=m, lens=[1000, m + 3], new=[m, m // 2], layout="paged", window=window, n_sink=n_sink, seed=3)
    c, t = CH.Case(**kw), Windowed(kind="chain", **kw)
    c.upload().call()
    t.upload()
    t.params["tree_window"] = True
    t.call()
    want = c.oracle()
    c.check(ora=want)
    t.check(ora=want)
