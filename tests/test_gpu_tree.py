"""kvsel_tree_masks and kvsel_attend_tree against the 64-bit oracle: trees from one node to many, every cache
layout, masks of any kind, windows, ragged batches, and calls that overlap or are captured."""
import numpy as np
import pytest

from oracle import step_oracle as SO
from tests import cache_harness as CH
from tests import step_harness as SH

pytestmark = pytest.mark.gpu
run = SH.run_tree


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    from kv_cache_eviction_window_gb300 import binding

    binding.load()
    yield


@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 64, 100, 257, 1024])
@pytest.mark.parametrize("kind", ["tree", "chain", "star"])
def test_masks(m, kind):
    import torch

    from kv_cache_eviction_window_gb300 import binding as L

    g = CH.rng(m)
    B, W = 3, -(-m // 32)
    new = [m, m // 2, 0]
    par = np.full((B, m), 5)
    for b in range(B):
        par[b, :new[b]] = SH.random_parents(g, new[b], kind)
    tree, pos = SH.ints(np.full((B, m, W), 9)), SH.ints(np.full((B, m), 9))
    L.kvsel_tree_masks(SH.ints(par), tree, pos=pos, first=SH.ints([10, 20, 30]), new_lens=SH.ints(new))
    tree, pos = tree.cpu().numpy().view(np.uint32), pos.cpu().numpy()
    for b in range(B):
        see = SO.ancestors(par[b, :new[b]].tolist())
        assert np.array_equal(tree[b, :new[b]], SO.words(see, m))
        assert np.array_equal(pos[b, :new[b]], 10 * (b + 1) + see.sum(axis=1) - 1)
        assert (tree[b, new[b]:] == 9).all() and (pos[b, new[b]:] == 9).all()
    # parents out of range are none; without positions and lengths
    odd = np.array([[5, -3, 2, 2, 3, 99, 1]])
    tree = torch.zeros((1, 7, 1), dtype=torch.int32, device="cuda")
    L.kvsel_tree_masks(SH.ints(odd), tree)
    assert np.array_equal(tree.cpu().numpy().view(np.uint32)[0], SO.words(SO.ancestors(odd[0].tolist()), 7))


@pytest.mark.parametrize("layout,block", [("contiguous", 0), ("packed", 0), ("paged", 8), ("paged", 16), ("paged", 32), ("paged", 64)])
@pytest.mark.parametrize("m,G", [(1, 1), (3, 4), (4, 4), (6, 5), (8, 4), (13, 7), (32, 4), (33, 4), (70, 4), (9, 16)])
def test_layouts_and_rows(layout, block, m, G):
    for n in (m, m + 1, 63 + m, 300, 700):
        if n >= m:
            run(layout=layout, block=block, lens=n, H=2, G=G, m=m, seed=n + m)


@pytest.mark.parametrize("m", [1, 2, 5, 17, 40, 65, 130])
@pytest.mark.parametrize("pad_rows", [0, 9000])
def test_lengths(m, pad_rows):
    # rows in use far below max_len too: the whole grid shares the work there
    for n in (m, m + 1, m + 62, m + 63, m + 64, m + 65, 1111):
        run(layout="paged", block=16, lens=n, H=2, G=4, m=m, pad_rows=pad_rows, seed=n)


@pytest.mark.parametrize("m,G", [(5, 2), (16, 4), (26, 7), (64, 4)])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (16, 0), (64, 4), (100, 70), (513, 4), (5000, 4)])
def test_windows(m, G, window, n_sink):
    run(B=2, layout="paged", block=8, lens=[1500, 140], H=2, G=G, m=m, window=window, n_sink=n_sink, seed=window)
    run(layout="contiguous", lens=900, H=2, G=G, m=m, window=window, n_sink=n_sink, seed=window + 1)


def test_ragged_batches():
    run(B=5, layout="paged", block=16, lens=[0, 1, 64, 513, 700], new=[0, 1, 16, 7, 3], m=16, G=4, seed=1)
    run(B=5, layout="paged", block=32, lens=[0, 40, 64, 5130, 700], new=[0, 40, 1, 33, 40], m=40, G=7, seed=2)
    run(B=3, layout="packed", lens=[[70, 300], [90, 40], [1000, 33]], new=[20, 33, 5], m=33, G=4, seed=3)
    run(B=3, layout="contiguous", lens=[[70, 300], [90, 40], [1000, 33]], new=[20, 33, 5], m=33, G=4, per_head=True, seed=4)
    run(B=4, layout="contiguous", lens=[200, 300, 9, 70], new=[8, 1, 2, 0], m=8, G=4, token_major=True, seed=5)
    run(B=2, layout="paged", lens=[3000, 77], new=[60, 20], m=60, G=8, token_major=True, scale=0.3, seed=6)


@pytest.mark.parametrize("m", [3, 20, 64, 150])
def test_any_mask(m):
    # masks that no tree has: bits at random, later nodes among them, and nodes that see nothing of the tree
    g = CH.rng(m)
    masks = [g.random((m, m)) < 0.3 for _ in range(2)]
    masks[0][m // 2] = False
    masks[1][:] = False
    run(B=2, lens=[m, 500], m=m, G=4, masks=masks, seed=m)              # (the first: a row that sees nothing)
    masks = [np.zeros((m, m), bool) for _ in range(2)]
    run(B=2, lens=m, m=m, G=4, masks=masks, seed=m)                     # no row sees anything
    run(B=2, lens=[400, 90 + m], m=m, G=4, window=32, n_sink=3, masks=[g.random((m, m)) < 0.1, np.zeros((m, m), bool)], seed=m)


@pytest.mark.parametrize("m,G", [(16, 4), (32, 4), (64, 8)])
def test_long_caches(m, G):
    run(lens=20011, H=1, G=G, m=m, layout="paged", block=64, seed=m)
    run(lens=8192, H=2, G=G, m=m, layout="contiguous", seed=m)


def test_a_chain_is_causal():
    # a chain's masks give what kvsel_attend gives
    c = CH.Case(B=2, H=2, G=4, m=24, lens=[1000, 77], new=[24, 11], layout="paged", seed=3)
    t = SH.TreeCase(B=2, H=2, G=4, m=24, lens=[1000, 77], new=[24, 11], layout="paged", seed=3, kind="chain")
    c.upload().call()
    t.upload().call()
    t.check(ora=c.oracle())


def test_rows_that_are_missing_from_the_cache():
    # fewer rows than nodes: the rows that are there belong to the last nodes
    masks = [np.tril(np.ones((8, 8), bool))]
    c = SH.TreeCase(lens=5, m=8, G=4, masks=masks)
    c.seen = lambda b, h: masks[0][:, 3:]
    c.seen_rows = lambda b, h: np.ones(5, bool)
    c.upload()
    assert CH.status(c.call()) == 0
    c.check()


def test_twice_the_same_bits_and_captured():
    import torch

    c = SH.TreeCase(B=3, H=4, G=4, m=32, lens=[3000, 511, 1], new=[32, 20, 1], layout="paged", seed=5).upload()
    ws = c.call()
    one = c.t["out"].clone()
    c.call(ws=ws)
    assert torch.equal(one, c.t["out"])
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            c.call(ws=ws, stream=torch.cuda.current_stream())
    torch.cuda.current_stream().wait_stream(s)
    # the captured call follows lengths and masks
    c.lens[0] = 2100
    c.t["lens"].copy_(SH.ints(c.lens[:, 0]))
    c.masks[0] = np.eye(32, dtype=bool)
    fresh = SH.TreeCase(B=3, H=4, G=4, m=32, lens=[2100, 511, 1], new=[32, 20, 1], layout="paged", seed=5, masks=c.masks,
                        pad_rows=900).upload()
    c.t["tree"].copy_(fresh.t["tree"])
    c.t["q"].copy_(fresh.t["q"])
    for a, b in zip(c.keep, fresh.keep):
        a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    c.check(ora=fresh.oracle())


def test_two_streams():
    import torch

    cases = [SH.TreeCase(B=2, H=4, G=4, m=m, lens=[2500, 300], layout="paged", seed=m).upload() for m in (4, 30, 64)]
    from kv_cache_eviction_window_gb300 import binding as L

    streams = [torch.cuda.Stream() for _ in cases]
    wss = [CH.workspace(L.kvsel_attend_tree_workspace_size(L.make_attn_params(**{**c.params, "acc_stride": 0}))) for c in cases]
    torch.cuda.synchronize()
    for c, s, ws in zip(cases, streams, wss):
        c.call(ws=ws, stream=s)
    for c, ws in zip(cases, wss):
        assert CH.status(ws) == 0
        c.check()


def test_bad_entries_are_recorded():
    c = SH.TreeCase(H=2, G=4, m=24, lens=300, layout="paged", seed=1).upload()
    c.keep[2][0, 3] = 10 ** 6
    assert CH.status(c.call()) == -7
    c = SH.TreeCase(H=2, G=4, m=24, lens=300, seed=1, new=[24]).upload()
    c.t["new_lens"][0] = 25
    assert CH.status(c.call()) == -7
    c.check()


def test_a_wait_that_runs_out():
    c = SH.TreeCase(H=2, G=4, m=64, lens=5000, layout="paged", seed=1).upload()
    c.params["wait_cycles"] = 1
    assert CH.status(c.call()) == -6
    c.params["wait_cycles"] = 0
    assert CH.status(c.call()) == 0
    c.check()
