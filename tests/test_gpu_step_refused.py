"""A step of drafted trees in which the pages do not suffice for every request: `granted` goes on as new_lens, and what
a refused request shares with others stays as it is."""
import numpy as np
import pytest

from oracle import step_oracle as SO
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


@pytest.mark.parametrize("spare,served", [(0, []), (1, [0]), (2, [0, 1, 2]), (3, [0, 1, 2, 3])])
@pytest.mark.parametrize("n_new", [9, 8192])         # (of the reservation: one launch, two)
def test_a_refused_request_takes_no_part(spare, served, n_new):
    # requests 0 to 2 share 37 rows in three pages, request 3 has a page of its own that is full; nine nodes each: copies of
    # the last page for 0 and 1, which 2 keeps, a page for 3
    import torch

    L, g = lib(), CH.rng(spare)
    B, m, H, G, bs, V, layers = 4, 9, 2, 4, 16, 50, 2
    table = np.array([[2, 5, 1, -1], [2, 5, 1, -1], [2, 5, 1, -1], [7, -1, -1, -1]])
    ref = np.array([1, 3, 3, 1, 1, 3, 1, 1, 1, 1])
    ref[[8, 0, 4][:spare]] = 0
    lens = np.array([37, 37, 37, 16])
    pool = [CH.bf16(g.standard_normal((layers, len(ref), bs, H, D))) for _ in range(2)]
    kd, vd = (CH.to_gpu_bf16(x) for x in pool)
    td, rd, ld, granted = SH.ints(table), SH.ints(ref), SH.ints(lens), SH.ints(np.full(B, 7))
    pp = L.make_pages_params(batch=B, max_blocks=4, num_blocks=len(ref), block_size=bs, h_kv=H, layers=layers, n_new=m)
    big = L.make_pages_params(batch=B, max_blocks=4, num_blocks=len(ref), block_size=bs, h_kv=H, layers=layers, n_new=n_new)
    ws = CH.workspace(1 << 24)
    nodes = SH.ints([m] * B)
    parents = np.array([SH.random_parents(g, m) for _ in range(B)])
    tokens = g.integers(V, size=(B, m))
    tree, pos = SH.ints(np.full((B, m, 1), 9)), SH.ints(np.full((B, m), 9))
    path, counts, nxt = SH.ints(np.full((B, m), 5)), SH.ints(np.full(B, 5)), SH.ints(np.full(B, 5))

    L.kvsel_pages_reserve(big, kd, vd, td, rd, ld, granted, ws, new_lens=nodes)
    want = [m if b in served else 0 for b in range(B)]
    assert granted.tolist() == want
    rows = ld + granted
    L.kvsel_tree_masks(SH.ints(parents), tree, pos=pos, first=ld, new_lens=granted)
    # the rows that this step may write: its requests' own pages
    at = td.cpu().numpy()
    fresh = [CH.bf16(g.standard_normal((layers, B, m, H, D))) for _ in range(2)]
    now = [x.copy() for x in pool]
    for b in served:
        if table[b, 2] >= 0 and at[b, 2] != table[b, 2]:
            for x in now:
                x[:, at[b, 2], :lens[b] % bs] = x[:, table[b, 2], :lens[b] % bs]
        assert int(rd[int(at[b, lens[b] // bs])]) == 1
        for x, y in zip(now, fresh):
            for t in range(m):
                j = lens[b] + t
                x[:, at[b, j // bs], j % bs] = y[:, b, t]
    for x, y, d in zip(now, fresh, (kd, vd)):
        for b in served:
            for t in range(m):
                j = lens[b] + t
                d[:, int(at[b, j // bs]), j % bs] = CH.to_gpu_bf16(y[:, b, t])
        assert np.array_equal(CH.to_f64(d)[:, ref > 0], x[:, ref > 0])           # (free pages may hold anything)
    q = CH.bf16(g.standard_normal((layers, B, H * G, m, D)))
    qd = CH.to_gpu_bf16(q)
    out = CH.to_gpu_bf16(np.full((layers, B, H * G, m, D), 7.0))
    pa = L.make_attn_params(h_kv=H, group=G, batch=B, n_new=m, max_len=4 * bs)
    for layer in range(layers):
        L.kvsel_attend_tree(pa, qd[layer], L.make_kv_paged(kd[layer], vd[layer], td), rows, tree, out[layer], ws, new_lens=granted)
    target = SH.probabilities(g, (B, m, V))
    draft = np.full((B, m, V), 1.0 / V, np.float32)
    u = g.random((B, m)).astype(np.float32)
    up = lambda x: torch.from_numpy(x).cuda()   # noqa: E731
    L.kvsel_verify(L.make_verify_params(batch=B, n_new=m, vocab=V), SH.ints(tokens), SH.ints(parents), up(target), path, counts, nxt, ws,
                   draft=up(draft), u=up(u), new_lens=granted)
    before = ld.tolist()
    L.kvsel_pages_accept(pp, kd, vd, td, rows, path, counts, ld, ws, new_lens=granted)
    L.kvsel_pages_trim(pp, td, rd, ld, ws)
    assert CH.status(ws) == 0

    got = CH.to_f64(out).reshape(layers, B, H, G, m, D)
    for b in range(B):
        if b not in served:
            assert (got[:, b] == 7.0).all() and int(counts[b]) == 0 and int(nxt[b]) == -1 and path[b].tolist() == [-1] * m
            assert int(ld[b]) == before[b] and td[b].tolist() == table[b].tolist() and (tree[b] == 9).all()
            continue
        see = SO.ancestors(parents[b].tolist())
        for layer in range(layers):
            k, v = (x[layer, at[b, :-(-(lens[b] + m) // bs)]].reshape(-1, H, D)[:lens[b] + m] for x in now)
            for h in range(H):
                o = SO.attend_seen(q[layer].reshape(B, H, G, m, D)[b, h], k[:, h], v[:, h], SO.tree_visible(lens[b] + m, see, 0, 0))
                e = (D + 4) * 2.0 ** -23 * o["abs_logit"] + 2.0 ** -14          # (as in the tests of the attention)
                tol = (2 * e[..., None] + 2.0 ** -8) * o["mean_abs"] + 2.0 ** -8 * np.abs(o["out"])
                assert np.all(np.abs(got[layer, b, h] - o["out"]) <= tol)
        nodes_, token = SO.verify(tokens[b].tolist(), parents[b].tolist(), target[b], draft[b], u[b], "sampled")
        assert path[b].tolist() == nodes_ + [-1] * (m - len(nodes_)) and int(nxt[b]) == token and int(ld[b]) == lens[b] + len(nodes_)
        for i, x in enumerate(nodes_):
            j0, j1 = lens[b] + x, lens[b] + i
            for y in now:
                y[:, at[b, j1 // bs], j1 % bs] = y[:, at[b, j0 // bs], j0 % bs]
    # pages that were in use hold what they held, but for the rows of requests that were served
    t2 = td.cpu().numpy()
    for x, d in zip(now, (kd, vd)):
        have = CH.to_f64(d)
        for b in range(B):
            n = int(ld[b])
            for j in range(n):
                assert np.array_equal(have[:, t2[b, j // bs], j % bs], x[:, t2[b, j // bs], j % bs]), (b, j)
        for page in (3, 6, 9):
            assert np.array_equal(have[:, page], x[:, page])
    uses = np.bincount(t2[t2 >= 0], minlength=len(ref))
    others = np.isin(np.arange(len(ref)), t2[t2 >= 0], invert=True) & (ref > 0) & ~np.isin(np.arange(len(ref)), table[table >= 0])
    assert np.array_equal(rd.cpu().numpy(), uses + others)
