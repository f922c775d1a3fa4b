"""Forms of kvsel_attend for few query rows under the bounds that are their own: weights that keep a
remainder, every cached row once, 17 to 32 query rows as two items, kept logits with several rows per thread."""
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


def few_rows(c):
    """Whether the call goes to the kernel of few rows: its partial results are 16 rows of 128 floats per CTA
    and slot, those of chunks at least 65 rows."""
    import torch

    from kv_cache_eviction_window_gb300 import binding as L

    sms = torch.cuda.get_device_properties(0).multi_processor_count
    size = L.kvsel_attend_workspace_size(L.make_attn_params(**c.params), False)
    return size < 70000 + 4 * sms * 16 * (512 + 8) + 4096


def run(c, acc=False, lse=True, tokens=True):
    c.upload()
    assert few_rows(c) == tokens
    ora = c.oracle()
    ws = c.call(acc=acc, lse=lse)
    assert CH.status(ws) == 0
    if lse:
        c.check(ora, acc=acc)
    if tokens:
        CH.check_tokens(c, ora)


# ------------------------------------------------------------------------------ the weights' remainder
@pytest.mark.parametrize("layout,block", [("contiguous", 0), ("packed", 0), ("paged", 8), ("paged", 64)])
@pytest.mark.parametrize("n", [1, 2, 3, 7, 16, 40, 64, 65, 130])
def test_weights_keep_a_remainder(layout, block, n):
    for pad in (0, 6000):       # an item to a cluster, and cut over the grid
        for m, G in ((1, 8), (2, 7), (1, 1)):
            run(CH.paired(CH.Case(layout=layout, block=block, lens=n, m=m, G=G, H=2, logit=0.1, pad_rows=pad, seed=n)))


# ------------------------------------------------------------------------------ every cached row, once
@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("kw", [
    dict(H=1, G=8, lens=20011), dict(H=2, G=4, lens=3001), dict(H=1, G=2, m=8, lens=12345, layout="paged", block=16),
    dict(H=3, G=5, B=2, lens=[[4099, 700, 64], [1, 2000, 333]], layout="packed"), dict(H=2, G=4, lens=9001, window=1000, n_sink=70),
    dict(H=2, G=4, lens=9001, window=5000, n_sink=4, layout="paged", block=64), dict(H=2, G=16, lens=1111, causal=False)])
def test_every_row_counts_once_for_tokens(kw, acc):
    run(CH.marked(CH.Case(scale=1e-3, seed=1, **kw)), acc=acc)


@pytest.mark.parametrize("kw", [
    dict(H=2, G=5, m=20, lens=12000), dict(H=2, G=4, m=130, lens=6000, layout="paged", block=16),
    dict(B=2, H=2, G=7, m=6, lens=[5001, 3000], layout="paged", block=32), dict(H=1, G=1, m=300, lens=20011),
    dict(B=2, H=2, G=4, m=70, lens=[9001, 300], window=3000, n_sink=70), dict(H=2, G=3, m=50, lens=4099, layout="packed"),
    dict(H=2, G=3, m=50, lens=4099, causal=False)])
def test_every_row_counts_once_for_chunks(kw):
    run(CH.marked(CH.Case(scale=1e-3, seed=1, **kw)), acc=True, tokens=False)


# ------------------------------------------------------------------------------ 17 to 32 query rows
TWO = [(3, 7), (4, 7), (1, 17), (1, 32), (6, 4), (8, 4), (17, 1), (2, 13)]


@pytest.mark.parametrize("m,G", TWO)
@pytest.mark.parametrize("layout,block", [("contiguous", 0), ("packed", 0), ("paged", 8), ("paged", 32)])
def test_two_items(m, G, layout, block):
    # clusters of one and of several, requests without tokens, with one, with all: an item that is empty, or
    # begins within a token's group
    for n in (1, 40, 100, 129, 500, 1111):
        for new in (None, [0, 1, m], [m, max(1, m - 1), 0]):
            lens = np.array([n, max(0, n - 9), n]) + (np.array([m] * 3) if new is None else np.array(new))
            run(CH.Case(B=3, H=2, G=G, m=m, lens=lens if layout != "packed" else np.repeat(lens[:, None], 2, 1), new=new,
                        layout=layout, block=block, token_major=n == 100, seed=n))


@pytest.mark.parametrize("m,G", TWO)
@pytest.mark.parametrize("layout,block", [("contiguous", 0), ("packed", 0), ("paged", 16)])
def test_two_items_with_windows(m, G, layout, block):
    for window, n_sink in ((1, 0), (2, 1), (40, 3), (130, 70), (700, 64)):
        for new in (None, [1, m]):
            lens = np.array([1201, m + 7])
            run(CH.Case(B=2, H=2, G=G, m=m, lens=lens if layout != "packed" else np.repeat(lens[:, None], 2, 1), new=new,
                        window=window, n_sink=n_sink, layout=layout, block=block, seed=window))


@pytest.mark.parametrize("m,G", TWO)
def test_two_items_of_every_kind(m, G):
    g = CH.rng(m)
    # every row visible; an empty cache; fewer rows than tokens; a length per head
    run(CH.Case(B=3, G=G, m=m, lens=[0, 77, 300], causal=False, new=[m, 1, m], seed=1))
    run(CH.Case(B=4, G=G, m=m, lens=[0, 1, m - 1, m], layout="paged", block=8, seed=2))
    run(CH.Case(B=2, H=4, G=G, m=m, lens=g.integers(m, 900, (2, 4)), per_head=True, layout="paged", block=16, seed=3))
    # as many segments as there are places for: clusters of one; and logits that make the maximum move
    run(CH.Case(B=9, H=8, G=G, m=m, lens=m + np.arange(9) * 12, seed=4))
    run(CH.Case(B=2, G=G, m=m, lens=[900, 321], scale=0.6, logit=3.0, seed=5))
    run(CH.paired(CH.Case(B=2, G=G, m=m, lens=[m + 5, 64], logit=0.1, seed=6)))
    run(CH.marked(CH.Case(H=1, G=G, m=m, lens=1500, scale=1e-3, seed=7)))
    run(CH.Case(B=2, G=G, m=m, lens=[m + 5, 640], seed=8), lse=False)


# ------------------------------------------------------------------------------ kept logits
@pytest.mark.parametrize("m,G", [(1, 4), (1, 3), (2, 2), (4, 1), (1, 1), (1, 8), (2, 4), (1, 5), (3, 2), (7, 1)])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (300, 5), (700, 300), (1, 0)])
def test_weights_of_many_rows(m, G, window, n_sink):
    """More than 1200 blocks of 256 rows: a thread adds up four cached rows (m G <= 7), or one."""
    lens = np.array([[255, 256, 257, 511, 513, 1023, 1025, 1], [0, 769, 767, 1279, 1281, 2047, 2100, 64],
                     [1536, 2049, 300, 900, 1793, 512, 768, 1024], [100, 1400, 1700, 2000, 258, 260, 514, 31]])
    for new in (None, [0, 1, m, m]):
        at = lens if new is None else np.maximum(lens, np.array(new)[:, None])
        c = CH.Case(B=4, H=8, G=G, m=m, lens=at, layout="packed", new=new, window=window, n_sink=n_sink, pad_rows=9000, seed=m)
        assert -(-c.max_len // 256) * 32 > 1200
        run(c, acc=True)


@pytest.mark.parametrize("m,G", [(1, 4), (2, 4)])
def test_weights_of_many_rows_from_pages(m, G):
    lens = 1200 - 37 * np.arange(20)
    for window, n_sink in ((0, 0), (333, 4)):
        run(CH.Case(B=20, H=8, G=G, m=m, lens=lens, layout="paged", block=16, window=window, n_sink=n_sink, pad_rows=849,
                    seed=window), acc=True)
    for calls in (1, 2):       # and they add up
        c = CH.Case(B=4, H=8, G=G, m=m, lens=[[2100, 900, 1025, 257, 1, 256, 0, 1999]] * 4, causal=False, layout="packed", pad_rows=9000, seed=3).upload()
        ws = None
        for _ in range(calls):
            ws = c.call(acc=True, ws=ws)
        assert CH.status(ws) == 0
        c.check(acc=True, calls=calls)
