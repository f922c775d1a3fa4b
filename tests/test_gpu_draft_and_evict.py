"""Drafted trees over a cache that is evicted from: rows of the tree by kvsel_evict_append, accepted ones by
kvsel_pages_accept, `seen` without the rejected ones, weights of the accepted tokens by kvsel_attend."""
import numpy as np
import pytest

from oracle import cache_oracle as CO
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


def close(got, o):
    # (the bound of the chunk kernel; that of the kernel of few rows is narrower)
    e = (D + 4) * 2.0 ** -23 * o["abs_logit"] + 2.0 ** -14
    tol = (2 * e[..., None] + 2.0 ** -8) * o["mean_abs"] + 2.0 ** -8 * np.abs(o["out"]) + 1e-30
    return bool(np.all(np.abs(got - o["out"]) <= tol))


@pytest.mark.parametrize("m,budget,spare", [(4, 60, 20), (9, 48, 20), (9, 48, 1), (33, 90, 20)])
def test_a_loop(m, budget, spare):
    import torch

    L, g = lib(), CH.rng(m)
    B, H, G, bs, V, start, sink, recent = 3, 2, 4, 16, 11, [40, 1, 25], 2, 12
    cap_pages = -(-(budget + m) // bs) + 1
    cap = cap_pages * bs
    total = sum(-(-n // bs) for n in start) + spare
    k, v = (CH.to_gpu_bf16(np.zeros((1, total, bs, H, D))) for _ in range(2))
    table, ref = SH.ints(np.full((B, cap_pages), -1)), SH.ints(np.zeros(total))
    d = dict(lens=SH.ints(np.zeros((B, H))), seen=SH.ints(np.zeros((B, H))), pos=SH.ints(np.zeros((B, H, cap))),
             acc=torch.zeros((B, H, cap), device="cuda"))
    kv = L.make_kv_paged(k[0], v[0], table)
    ws = CH.workspace(1 << 27)
    granted = SH.ints(np.zeros(B))

    def append(n_new, new):
        pp = L.make_pages_params(batch=B, max_blocks=cap_pages, num_blocks=total, block_size=bs, h_kv=H, n_new=n_new, lens_per_head=True)
        pe = L.make_evict_params(h_kv=H, batch=B, capacity=cap, budget=budget, n_new=n_new, n_sink=sink, n_recent=recent)
        kn, vn = (CH.bf16(g.standard_normal((B, H, n_new, D))) for _ in range(2))
        L.kvsel_pages_reserve(pp, k, v, table, ref, d["lens"], granted, ws, new_lens=SH.ints(new))
        L.kvsel_evict_append(pe, kv, d["lens"], d["seen"], d["pos"], d["acc"], CH.to_gpu_bf16(kn), CH.to_gpu_bf16(vn), ws, new_lens=granted)
        return pp, kn, vn, granted.tolist()

    # the state here: rows, positions and weights of every segment
    rows = {(b, h): (np.zeros((0, D)), np.zeros((0, D)), np.zeros(0, int), np.zeros(0)) for b in range(B) for h in range(H)}
    seen = [0] * B

    def appended(kn, vn, new):
        for (b, h), (rk, rv, pos, acc) in rows.items():
            x = new[b]
            order = CO.evict_segment(pos, acc.astype(np.float32), seen[b], x, budget=budget, n_sink=sink, n_recent=recent)
            rows[b, h] = (np.concatenate([rk[order], kn[b, h, :x]]), np.concatenate([rv[order], vn[b, h, :x]]),
                          np.concatenate([pos[order], seen[b] + np.arange(x)]), np.concatenate([acc[order], np.zeros(x)]))
        for b in range(B):
            seen[b] += new[b]

    def weigh(counts, q):
        """kvsel_attend with weights for the last counts[b] rows; queries [B][H*G][..][D]."""
        n_new = q.shape[2]
        pa = L.make_attn_params(h_kv=H, group=G, batch=B, n_new=n_new, max_len=cap, lens_per_head=True, acc_stride=cap)
        out = CH.to_gpu_bf16(np.zeros((B, H * G, n_new, D)))
        L.kvsel_attend(pa, CH.to_gpu_bf16(q), kv, d["lens"], out, ws, new_lens=SH.ints(counts), acc=d["acc"])
        got, da = CH.to_f64(out).reshape(B, H, G, n_new, D), d["acc"].cpu().numpy()
        for (b, h), (rk, rv, pos, acc) in rows.items():
            if counts[b]:
                o = CO.attend_segment(q.reshape(B, H, G, n_new, D)[b, h, :, :counts[b]], rk, rv)
                assert close(got[b, h, :, :counts[b]], o)
                e = (D + 4) * 2.0 ** -23 * o["abs_logit"] + 2.0 ** -14
                # (a sum onto what was there: one more rounding of each)
                tol = (2 * e.max() + (G * counts[b] + 2) * 2.0 ** -23) * o["weight"] + 2.0 ** -23 * (acc + o["weight"]) + 1e-30
                assert np.all(np.abs(da[b, h, :len(acc)] - (acc + o["weight"])) <= tol)
            # (its rounding decides the next eviction)
            rows[b, h] = (rk, rv, pos, da[b, h, :len(acc)].astype(np.float64))
        return got

    _, kn, vn, new = append(max(start), start)
    assert new == start
    appended(kn, vn, new)
    weigh(start, CH.bf16(g.standard_normal((B, H * G, max(start), D))))
    refused = evicted = 0
    for step in range(30):
        nodes = [m if step % 3 else int(g.integers(0, m + 1)) for _ in range(B)]
        before = [sum(len(rows[b, h][2]) for h in range(H)) for b in range(B)]
        pp, kn, vn, new = append(m, nodes)
        refused += sum(x < y for x, y in zip(new, nodes))
        appended(kn, vn, new)
        evicted += sum(sum(len(rows[b, h][2]) for h in range(H)) < before[b] + H * new[b] for b in range(B))
        parents = np.array([SH.random_parents(g, m) for _ in range(B)])
        tokens = g.integers(V, size=(B, m))
        q = CH.bf16(g.standard_normal((B, H * G, m, D)))
        tree = SH.ints(np.zeros((B, m, -(-m // 32))))
        out = CH.to_gpu_bf16(np.full((B, H * G, m, D), 7.0))
        path, counts, nxt = SH.ints(np.zeros((B, m))), SH.ints(np.zeros(B)), SH.ints(np.zeros(B))
        L.kvsel_tree_masks(SH.ints(parents), tree, new_lens=granted)
        pa = L.make_attn_params(h_kv=H, group=G, batch=B, n_new=m, max_len=cap, lens_per_head=True)
        L.kvsel_attend_tree(pa, CH.to_gpu_bf16(q), kv, d["lens"], tree, out, ws, new_lens=granted)
        logits = g.standard_normal((B, m, V)).astype(np.float32)
        L.kvsel_verify(L.make_verify_params(batch=B, n_new=m, vocab=V, mode="greedy"), SH.ints(tokens), SH.ints(parents),
                       torch.from_numpy(logits).cuda(), path, counts, nxt, ws, new_lens=granted)
        L.kvsel_pages_accept(pp, k, v, table, d["lens"], path, counts, d["lens"], ws, new_lens=granted)
        L.kvsel_pages_trim(pp, table, ref, d["lens"], ws)
        d["seen"] -= (granted - counts)[:, None]
        assert CH.status(ws) == 0
        got = CH.to_f64(out).reshape(B, H, G, m, D)
        line = [SO.verify(tokens[b, :new[b]].tolist(), parents[b].tolist(), logits[b], None, None, "greedy")[0] for b in range(B)]
        assert [[x for x in r if x >= 0] for r in path.tolist()] == line
        for (b, h), (rk, rv, pos, acc) in rows.items():
            n, x = len(rk), new[b]
            if x:
                o = SO.attend_seen(q.reshape(B, H, G, m, D)[b, h, :, :x], rk, rv, SO.tree_visible(n, SO.ancestors(parents[b, :x].tolist()), 0, 0))
                assert close(got[b, h, :, :x], o)
            stay = list(range(n - x)) + [n - x + t for t in line[b]]
            c = len(line[b])
            # accepted rows: the places of the first ones, whose pos and acc are theirs
            rows[b, h] = (rk[stay], rv[stay], pos[:n - x + c], acc[:n - x + c])
        seen = [s - new[b] + len(line[b]) for b, s in enumerate(seen)]
        n_max = max(map(len, line))
        if n_max:
            qa = np.zeros((B, H * G, n_max, D))
            for b in range(B):
                qa[b, :, :len(line[b])] = q[b][:, line[b]]
            weigh([len(x) for x in line], qa)
        assert CH.status(ws) == 0
        dl, ds, dp, t = (x.cpu().numpy() for x in (d["lens"], d["seen"], d["pos"], table))
        kh, vh = CH.to_f64(k[0]), CH.to_f64(v[0])
        for (b, h), (rk, rv, pos, acc) in rows.items():
            n = len(rk)
            assert dl[b, h] == n <= budget and ds[b, h] == seen[b] and np.array_equal(dp[b, h, :n], pos)
            j = np.arange(n)
            assert np.array_equal(kh[t[b, j // bs], j % bs, h], rk) and np.array_equal(vh[t[b, j // bs], j % bs, h], rv)
        assert int(ref.sum()) == int((t >= 0).sum())
    assert evicted > 0 and (refused > 0) == (spare == 1)
