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
