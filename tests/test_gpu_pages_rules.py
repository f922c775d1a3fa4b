"""Reservations of pages that have to be refused in part: lengths that no cache has, entries that no table has."""
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


def lib():
    from kv_cache_eviction_window_gb300 import binding

    return binding


def guarded(c):
    """The table between words that name pages in use, so that a row before or behind it would be served or refused by
    what lies there."""
    import torch

    B, cap = c.table.shape
    wide = torch.full((B * cap + 128,), int(c.table.max()), dtype=torch.int32, device="cuda")
    wide[64:-64] = c.table.reshape(-1)
    c.table = wide[64:-64].view(B, cap)
    return wide


@pytest.mark.parametrize("n_new", [64, 8192])        # (one launch; two, with pages of 8)
@pytest.mark.parametrize("bs", [8, 64])
@pytest.mark.parametrize("where", [0, 1, 2])
@pytest.mark.parametrize("length", [-1, -8, -1000, -2 ** 31])
def test_a_negative_length_is_recorded_and_the_others_are_served(n_new, bs, where, length):
    c = SH.PageCase(B=3, bs=bs, rows=[20, 33, 70], cap=16, spare=30, seed=bs).upload()
    wide = guarded(c)
    before, granted = wide.clone(), SH.ints([7, 7, 7])
    c.d_lens[where] = length
    lib().kvsel_pages_reserve(c.params(n_new), c.k, c.v, c.table, c.ref, c.d_lens, granted, c.ws, new_lens=SH.ints([9, 9, 9]))
    assert CH.status(c.ws) == -7
    new = [9, 9, 9]
    new[where] = 0
    assert np.array_equal(c.o.reserve(c.lens, new), granted.cpu().numpy())
    c.check()
    assert wide[:64].equal(before[:64]) and wide[-64:].equal(before[-64:])


@pytest.mark.parametrize("n_new", [64, 8192])
@pytest.mark.parametrize("length", [-1, -2 ** 31])
def test_a_negative_length_of_one_head(n_new, length):
    c = SH.PageCase(B=2, H=3, bs=8, rows=[[5, 20, 33], [16, 16, 0]], per_head=True, cap=16, spare=30, seed=2).upload()
    guarded(c)
    granted = SH.ints([7, 7])
    c.d_lens[0, 1] = length
    lib().kvsel_pages_reserve(c.params(n_new), c.k, c.v, c.table, c.ref, c.d_lens, granted, c.ws, new_lens=SH.ints([4, 4]))
    assert CH.status(c.ws) == -7
    assert np.array_equal(c.o.reserve(c.lens, [0, 4]), granted.cpu().numpy())
    c.check()


@pytest.mark.parametrize("n_new", [64, 8192])
@pytest.mark.parametrize("entry", [-2, -2 ** 31, 10 ** 6])
def test_an_entry_that_no_table_has(n_new, entry):
    c = SH.PageCase(B=3, bs=8, rows=[20, 20, 20], cap=8, spare=30, seed=1).upload()
    granted, was = SH.ints([7, 7, 7]), c.table[1].clone()
    c.table[1, 3] = entry
    lib().kvsel_pages_reserve(c.params(n_new), c.k, c.v, c.table, c.ref, c.d_lens, granted, c.ws, new_lens=SH.ints([9, 9, 9]))
    assert CH.status(c.ws) == -7
    assert c.o.reserve(c.lens, [9, 0, 9]).tolist() == granted.tolist() and int(c.table[1, 3]) == entry
    c.table[1] = was
    c.check()


@pytest.mark.parametrize("spare", [200, 9000, 13000])
def test_thousands_of_shared_pages(spare):
    # beams of four that set their lengths back: all their pages are shared, and new rows go to all of them
    B, pages = 64, 256
    share = [None if b % 4 == 0 else b - b % 4 for b in range(B)]
    c = SH.PageCase(B=B, H=1, L=1, bs=8, rows=[8 * pages] * B, cap=pages + 4, spare=spare, share=share, seed=spare)
    c.o.ref[np.flatnonzero(c.o.ref == 0)[spare:]] = 1   # (free pages: as many as are left so)
    c.upload()
    c.lens[:] = [3 + b for b in range(B)]
    c.d_lens.copy_(SH.ints(c.lens))
    new = [8 * pages - 3 - b if b % 7 else 5 for b in range(B)]
    granted = SH.ints([7] * B)
    for turn in range(2):                            # (and again: what is reserved already stays)
        lib().kvsel_pages_reserve(c.params(8 * pages), c.k, c.v, c.table, c.ref, c.d_lens, granted, c.ws, new_lens=SH.ints(new))
        assert CH.status(c.ws) == 0
        assert np.array_equal(c.o.reserve(c.lens, new), granted.cpu().numpy())
        c.check()
    assert (spare > 12288) == all(granted.tolist())


@pytest.mark.parametrize("n_new", [64, 8192])
@pytest.mark.parametrize("gap", [0, 8])              # K and V of a layer side by side; elements between layers beside them
def test_layers_further_apart_than_they_are_long(n_new, gap):
    import torch

    c = SH.PageCase(B=4, H=2, L=5, rows=[21, 21, 40, 16], share=[None, 0, None, None], cap=12, spare=30, seed=5).upload()
    layer = c.k[0].numel()
    stride = 2 * layer + gap
    wide = torch.full((5, stride), 77, dtype=torch.int16, device="cuda")
    k, v = (wide[:, i * layer:(i + 1) * layer].unflatten(1, c.k.shape[1:]) for i in range(2))
    k.copy_(c.k)
    v.copy_(c.v)

    def params(n):
        return lib().make_pages_params(batch=4, max_blocks=12, num_blocks=len(c.o.ref), block_size=16, h_kv=2, layers=5, n_new=n, stride_layer=stride)

    granted, new = SH.ints([7] * 4), [9, 3, 9, 1]
    lib().kvsel_pages_reserve(params(n_new), k, v, c.table, c.ref, c.d_lens, granted, c.ws, new_lens=SH.ints(new))
    assert np.array_equal(c.o.reserve(c.lens, new), granted.cpu().numpy())
    paths = [[0, 4, 8], [0], [0, 1, 2, 7], []]
    path, out = np.full((4, 9), -1), SH.ints([0] * 4)
    for b, x in enumerate(paths):
        path[b, :len(x)] = x
    rows = c.lens + new
    lib().kvsel_pages_accept(params(9), k, v, c.table, SH.ints(rows), SH.ints(path), SH.ints([len(x) for x in paths]), out, c.ws,
                             new_lens=SH.ints(new))
    assert CH.status(c.ws) == 0
    assert np.array_equal(c.o.accept(rows, new, paths), out.cpu().numpy())
    c.k, c.v = k.contiguous(), v.contiguous()
    c.check()
    assert bool((wide[:, 2 * layer:] == 77).all())
