"""Ends of the ranges that a step of drafted tokens allows: the largest trees and groups, pools and probabilities past
2^32 elements, many requests, heads that keep different numbers of rows, and calls from a new host thread."""
import threading

import numpy as np
import pytest

from tests import cache_harness as CH
from tests import step_harness as SH

pytestmark = pytest.mark.gpu
D = CH.D


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    yield


def lib():
    from kv_cache_eviction_window_gb300 import binding

    return binding


@pytest.mark.parametrize("m,G,n,layout", [(1024, 1, 1500, "paged"), (1024, 2, 1024, "contiguous"), (300, 16, 700, "paged"),
                                          (5, 128, 300, "paged"), (130, 5, 2000, "packed"), (1, 128, 5000, "paged")])
def test_large_trees_and_groups(m, G, n, layout):
    SH.run_tree(H=1, G=G, m=m, lens=n, layout=layout, block=16, seed=m)


def test_many_requests():
    # more items than CTAs, of every kind of work
    SH.run_tree(B=100, H=2, G=4, m=6, lens=[7 + 11 * (i % 40) for i in range(100)], new=[i % 7 for i in range(100)], layout="paged", seed=1)
    SH.run_tree(B=100, H=2, G=4, m=40, lens=[40 + 11 * (i % 40) for i in range(100)], new=[(i * 7) % 41 for i in range(100)], layout="paged", seed=2)
    SH.run_tree(B=300, H=1, G=2, m=3, lens=[3 + i for i in range(300)], layout="contiguous", seed=3)


@pytest.mark.parametrize("m,G,long", [(8, 4, 500), (8, 4, 4000), (50, 4, 300), (50, 4, 4000), (4, 32, 900), (70, 2, 4100)])
def test_more_items_than_ctas(m, G, long):
    # whole items in waves, or cut ones where some are long; requests without nodes or rows among them
    lens = [long if i == 77 else (i * 13) % 180 for i in range(200)]
    SH.run_tree(B=200, H=1, G=G, m=m, lens=lens, new=[min(n, (i * 7) % (m + 1)) for i, n in enumerate(lens)], layout="paged", block=16, seed=m)
    SH.run_tree(B=200, H=1, G=G, m=m, lens=lens, new=[min(n, m) for n in lens], layout="contiguous", window=90, n_sink=3, seed=m + 1)


@pytest.mark.parametrize("B", [1, 500, 700])
def test_many_requests_and_pages(B):
    # (up to 1024 touched entries in one launch, more in two)
    share = [None if i % 5 == 0 else i - i % 5 for i in range(B)]
    c = SH.PageCase(B=B, H=1, L=2, bs=8, rows=[8 * (i // 5 % 4) + i // 5 % 8 for i in range(B)], cap=8, spare=2 * B + 40, share=share, seed=B).upload()
    p, granted = c.params(1), SH.ints(np.zeros(B))
    lib().kvsel_pages_reserve(p, c.k, c.v, c.table, c.ref, c.d_lens, granted, c.ws)
    assert CH.status(c.ws) == 0
    assert np.array_equal(c.o.reserve(c.lens, [1] * B), granted.cpu().numpy())
    c.check()
    src, out = c.g.permutation(B), SH.ints(np.zeros(B))
    lib().kvsel_pages_fork(p, c.table, c.d_lens, SH.ints(src), c.other, out, c.ref, c.ws)
    c.o.fork(src.tolist())
    assert CH.status(c.ws) == 0
    c.check(c.other)


def test_pools_past_two_to_the_32():
    # 270,000 pages of 16 rows x 8 heads: 4.4e9 elements a side; the pages in use are the last ones
    import torch

    L, N, bs, H = lib(), 270000, 16, 8
    k, v = (torch.empty((1, N, bs, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ref = torch.ones(N, dtype=torch.int32, device="cuda")
    ref[N - 20:] = 0
    table = SH.ints([[N - 1, N - 2, -1, -1], [N - 1, N - 3, -1, -1]])
    ref[N - 1], ref[N - 2], ref[N - 3] = 2, 1, 1
    g = CH.rng(1)
    rows = CH.to_gpu_bf16(CH.bf16(g.standard_normal((2, 3, bs, H, D))))
    for x, r in ((k, rows[0]), (v, rows[1])):
        x[0, N - 3:] = r
    p = L.make_pages_params(batch=2, max_blocks=4, num_blocks=N, block_size=bs, h_kv=H, n_new=4)
    ws, granted, lens = CH.workspace(L.kvsel_pages_workspace_size(p)), SH.ints([0, 0]), SH.ints([9, 30])
    # request 0 writes to the shared page: a copy in the lowest free page; request 1 gets one more page
    L.kvsel_pages_reserve(p, k, v, table, ref, lens, granted, ws)
    assert CH.status(ws) == 0 and granted.tolist() == [4, 4]
    assert table.tolist() == [[N - 20, N - 2, -1, -1], [N - 1, N - 3, N - 19, -1]]
    assert torch.equal(k[0, N - 20, :9], rows[0, 2, :9]) and torch.equal(v[0, N - 20, :9], rows[1, 2, :9])
    # accepted rows: rows 30, 31 of page N - 3, 32, 33 of page N - 19
    fresh = CH.to_gpu_bf16(CH.bf16(g.standard_normal((2, 2, H, D))))
    k[0, N - 19, :2], v[0, N - 19, :2] = fresh[0], fresh[1]
    L.kvsel_pages_accept(p, k, v, table, SH.ints([13, 34]), SH.ints([[0, -1, -1, -1], [0, 2, 3, -1]]), SH.ints([1, 3]), lens, ws)
    assert CH.status(ws) == 0 and lens.tolist() == [10, 33]
    assert torch.equal(k[0, N - 3, 15], fresh[0, 0]) and torch.equal(v[0, N - 19, 0], fresh[1, 1])
    # kept rows of one request, and its keys turned
    kv = L.make_kv_paged(k[0], v[0], table[1:2, :2].contiguous())
    q = L.make_params(h_kv=H, group=1, n_ctx=32, window=32, n_ctx_per_req=[32], n_sink=0, n_recent=0, budget_ratio=0.25)
    idx = SH.ints(np.tile([1, 3, 5, 20, 24, 29, 30, 31], (H, 1)))
    before = torch.cat([k[0, N - 1], k[0, N - 3]])
    pos = SH.ints(np.zeros((1, H, 32)))
    L.kvsel_compact_in_place(q, kv, idx, SH.ints([8] * H), torch.arange(H, device="cuda") * 8, SH.ints([0] * H), None, pos, ws)
    assert CH.status(ws) == 0
    where = [20, 1, 24, 3, 29, 5, 30, 31]
    assert pos[0, 0, :8].tolist() == where and torch.equal(k[0, N - 1, :8], before[where])
    t = L.kvsel_rope_table()
    out = CH.to_gpu_bf16(np.zeros((1, H, 8, D)))
    L.kvsel_rope_cache(t, kv, SH.ints([8]), SH.ints(np.zeros((1, H, 8))), ws, out=out)
    assert CH.status(ws) == 0 and torch.equal(out[0].transpose(0, 1), k[0, N - 1, :8])


def test_probabilities_past_two_to_the_32():
    # 300 requests of 128 nodes over 131072 tokens: 5.0e9 values; the last request walks a chain
    import torch

    L, B, m, V = lib(), 300, 128, 131072
    target = torch.zeros((B, m, V), dtype=torch.bfloat16, device="cuda")
    tokens = np.zeros((B, m), int)
    parents = np.tile(np.arange(-1, m - 1), (B, 1))
    want = [(t * 977) % V for t in range(m)]
    for t in range(m):
        target[B - 1, t, want[t]] = 1.0
    tokens[B - 1, 1:100] = want[:99]
    tokens[B - 1, 100] = want[99] + 1
    ws = CH.workspace(1 << 17)
    for mode in ("greedy", "point"):
        path, counts, nxt = SH.ints(np.zeros((B, m))), SH.ints(np.zeros(B)), SH.ints(np.zeros(B))
        L.kvsel_verify(L.make_verify_params(batch=B, n_new=m, vocab=V, mode=mode, dtype="bf16"), SH.ints(tokens), SH.ints(parents), target, path,
                       counts, nxt, ws, u=None if mode == "greedy" else torch.full((B, m), 0.5, device="cuda"))
        assert CH.status(ws) == 0
        assert counts.tolist()[B - 1] == 100 and path[B - 1].tolist() == list(range(100)) + [-1] * 28 and nxt.tolist()[B - 1] == want[99]
        # the others: token 0 is the largest of equal values, or has no mass
        assert counts.tolist()[0] == (m if mode == "greedy" else 1) and nxt.tolist()[0] == (0 if mode == "greedy" else -1)


def test_heads_that_keep_different_numbers():
    # one budget for the layer: what kvsel_compact gathers, found in place
    import torch

    L, B, H, lens = lib(), 3, 4, [700, 64, 333]
    g = CH.rng(3)
    p = L.make_params(h_kv=H, group=1, n_ctx=700, window=32, n_ctx_per_req=lens, n_sink=2, n_recent=8, budget_mode="layer", budget_ratio=0.3)
    n_scores, n_kept, n_seg = L.kvsel_output_size(p)
    scores = torch.from_numpy((np.exp(g.standard_normal(n_scores)) * np.repeat(np.arange(1, n_seg + 1), np.repeat(lens, H))).astype(np.float32)).cuda()
    k, v = (CH.to_gpu_bf16(CH.bf16(g.standard_normal((B, H, 700, D)))) for _ in range(2))
    kv = L.make_kv_contiguous(k, v)
    idx, counts, offsets = SH.ints(np.zeros(n_kept)), SH.ints(np.zeros(n_seg)), torch.zeros(n_seg, dtype=torch.int64, device="cuda")
    ws = CH.workspace(max(1 << 20, L.kvsel_workspace_size(p)))
    L.kvsel_select(p, scores, None, idx, counts, offsets, ws)
    ko, vo = (torch.zeros((n_kept, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    L.kvsel_compact(p, kv, idx, counts, offsets, ko, vo, ws)
    lens_out, pos = SH.ints(np.zeros((B, H))), SH.ints(np.full((B, H, 700), -1))
    L.kvsel_compact_in_place(p, kv, idx, counts, offsets, lens_out, None, pos, ws)
    assert CH.status(ws) == 0 and torch.equal(lens_out.flatten(), counts) and len(set(counts.tolist())) > 1
    for s, (c, o) in enumerate(zip(counts.tolist(), offsets.tolist())):
        b, h = divmod(s, H)
        order = torch.argsort(pos[b, h, :c])
        assert torch.equal(pos[b, h, :c][order], idx[o:o + c])
        assert torch.equal(k[b, h, :c][order], ko[o:o + c]) and torch.equal(v[b, h, :c][order], vo[o:o + c])


@pytest.mark.parametrize("B,n,hq,hk", [(1, 3, 300, 5), (1000, 1, 2, 1), (1, 40000, 2, 0)])
def test_rows_of_many_heads_requests_and_tokens(B, n, hq, hk):
    from tests import test_gpu_rope as TR

    t, o = TR.table(layout="interleaved")
    g = CH.rng(n)
    x, pos = CH.bf16(g.standard_normal((B, hq + hk, n, D))), g.integers(0, 10 ** 6, (B, n))
    q = CH.to_gpu_bf16(x)
    lib().kvsel_rope(t, q[:, :hq], SH.ints(pos), k=q[:, hq:] if hk else None)
    TR.close(CH.to_f64(q), x, pos[:, None], o)


def test_from_a_new_host_thread():
    import torch

    fails = []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                c = SH.TreeCase(H=2, G=4, m=24, lens=300, layout="paged", seed=1).upload()
                assert CH.status(c.call()) == 0
                c.check()
                v = SH.VerifyCase(B=2, m=6, V=500, seed=1).upload()
                assert CH.status(v.call()) == 0
                v.check()
        except BaseException as e:      # noqa: BLE001 - handed to the test
            fails.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not fails, fails
