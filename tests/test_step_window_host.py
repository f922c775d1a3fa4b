"""A window that counts the tree's own rows: the oracle's rule by hand, by depth and against causal attention; refusals."""
import numpy as np
import pytest

from oracle import cache_oracle as CO
from oracle import step_oracle as SO
from tests import cache_harness as CH
from tests import step_harness as SH


@pytest.mark.parametrize("n,m,window,sink", [(20, 8, 4, 0), (20, 8, 1, 0), (20, 8, 4, 2), (12, 8, 3, 6), (8, 8, 3, 2), (8, 8, 8, 0), (20, 8, 0, 0),
                                             (5, 8, 3, 0), (5, 8, 3, 4), (1024, 1024, 512, 4)])
def test_a_chain_is_causal(n, m, window, sink):
    chain = SO.ancestors([t - 1 for t in range(m)])
    assert np.array_equal(SO.tree_windowed(n, chain, window, sink), CO.visible(n, m, True, window, sink))


def test_by_hand():
    see = SO.ancestors([-1, 0, 0, 1, 2])
    # seven rows, the last five the tree's.  Nodes 3 and 4 are at position 4 and see the last two positions: 3 and 4, their
    # parents' and their own; with one first row that too
    assert SO.tree_windowed(7, see, 2, 0).astype(int).tolist() == [
        [0, 1, 1, 0, 0, 0, 0], [0, 0, 1, 1, 0, 0, 0], [0, 0, 1, 0, 1, 0, 0], [0, 0, 0, 1, 0, 1, 0], [0, 0, 0, 0, 1, 0, 1]]
    assert SO.tree_windowed(7, see, 2, 1)[3].astype(int).tolist() == [1, 0, 0, 1, 0, 1, 0]
    # first rows that reach into the tree: positions 0 to 2
    assert SO.tree_windowed(7, see, 1, 3)[3].astype(int).tolist() == [1, 1, 1, 0, 0, 1, 0]


@pytest.mark.parametrize("seed", range(6))
def test_by_depth(seed):
    g = CH.rng(seed)
    m, n, window, sink = 40, 40 + int(g.integers(0, 5)), int(g.integers(1, 8)), int(g.integers(0, 7))
    par = SH.random_parents(g, m)
    depth = [0]
    for t in range(1, m):
        depth.append(depth[par[t]] + 1)
    see, got = SO.ancestors(par), SO.tree_windowed(n, SO.ancestors(par), window, sink)
    base = n - m
    for t in range(m):
        for u in range(m):
            near = depth[t] - depth[u] < window or base + depth[u] < sink
            assert got[t, base + u] == (see[t, u] and near)
        for j in range(base):
            assert got[t, j] == (base + depth[t] - j < window or j < sink)


def test_refusals():
    import __graft_entry__

    __graft_entry__.build()
    from kv_cache_eviction_window_gb300 import binding as L

    for x in (-1, 2):
        p = L.make_attn_params(h_kv=2, group=4, batch=1, max_len=100, window=3)
        p.tree_window = x
        with pytest.raises(L.KvselError) as e:
            L.kvsel_attend_tree_workspace_size(p)
        assert e.value.code == -1
    p = L.make_attn_params(h_kv=2, group=4, batch=1, max_len=100, window=3, tree_window=True)
    assert p.tree_window == 1 and L.make_attn_params(h_kv=2, group=4, batch=1, max_len=100).tree_window == 0
