"""The calls of a step of drafted tokens together, as a decode loop makes them: masks and positions, rotation, rows
appended to reserved pages, attention of the tree, verification, accepted rows, freed pages; and a selection that
stays in its cache, goes on with eviction and attention, and gives its pages back."""
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


class Loop:
    """Requests that share a prompt's pages, two layers, a toy model: rows of q, k and v by token and layer, rotated
    by position; the next token's probabilities from the attention's output."""

    def __init__(self, B, m, prompt, seed, captured=False):
        import torch

        L = lib()
        self.B, self.m, self.H, self.G, self.layers, self.bs, self.V = B, m, 2, 4, 2, 16, 97
        g = self.g = CH.rng(seed)
        new = lambda *s: CH.to_gpu_bf16(CH.bf16(g.standard_normal(s)))   # noqa: E731
        self.emb_q, self.emb_k, self.emb_v = new(self.layers, self.V, self.H * self.G, D), new(self.layers, self.V, self.H, D), new(self.layers, self.V, self.H, D)
        self.head = torch.from_numpy(g.standard_normal((self.V, D)).astype(np.float32)).cuda() * 1.5
        self.cap, total = 40, 400
        self.k, self.v = (torch.zeros((self.layers, total, self.bs, self.H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.table = SH.ints(np.full((B, self.cap), -1))
        self.other = SH.ints(np.full((B, self.cap), -1))
        self.ref, self.lens, self.lens2 = SH.ints(np.zeros(total)), SH.ints(np.zeros(B)), SH.ints(np.zeros(B))
        self.granted, self.counts, self.next = (SH.ints(np.zeros(B)) for _ in range(3))
        self.path = SH.ints(np.zeros((B, m)))
        self.tree, self.pos = SH.ints(np.zeros((B, m, -(-m // 32)))), SH.ints(np.zeros((B, m)))
        self.turn = L.kvsel_rope_table(theta=500000.0, scaling="bands", factor=8.0, orig_len=64)
        self.ws = CH.workspace(1 << 24)
        self.texts = None
        # the prompt, once, for request 0; the others fork it
        self.prompt = g.integers(self.V, size=prompt).tolist()
        p = self.params(prompt)
        one = SH.ints([prompt] + [0] * (B - 1))
        L.kvsel_pages_reserve(p, self.k, self.v, self.table, self.ref, self.lens, self.granted, self.ws, new_lens=one)
        self.lens.copy_(one)
        self.write(0, 0, self.prompt, range(prompt))
        L.kvsel_pages_fork(p, self.table, self.lens, SH.ints([0] * B), self.other, self.lens2, self.ref, self.ws)
        self.table, self.other, self.lens, self.lens2 = self.other, self.table, self.lens2, self.lens
        self.texts = [list(self.prompt) for _ in range(B)]
        assert CH.status(self.ws) == 0

    def params(self, n_new):
        return lib().make_pages_params(batch=self.B, max_blocks=self.cap, num_blocks=len(self.ref), block_size=self.bs, h_kv=self.H,
                                       layers=self.layers, n_new=n_new)

    def turned(self, x, positions):
        """Rows [layers][heads][tokens][d] by kvsel_rope."""
        y = x.clone()
        lib().kvsel_rope(self.turn, y, SH.ints(positions))
        return y

    def write(self, b, start, tokens, positions):
        """Rows of tokens at rows start.. of request b, in every layer (what a model's projections would do)."""
        import torch

        t = torch.tensor(tokens, device="cuda")
        k = self.turned(self.emb_k[:, t].transpose(1, 2).contiguous(), np.asarray(positions))
        v = self.emb_v[:, t].transpose(1, 2)
        rows = torch.arange(start, start + len(tokens), device="cuda")
        page, slot = self.table[b].long()[rows // self.bs], rows % self.bs
        assert bool((page >= 0).all()) and bool((self.ref[page] == 1).all())     # its own to write
        for pool, x in ((self.k, k), (self.v, v)):
            pool[:, page, slot] = x.transpose(1, 2)

    def step(self, new):
        import torch

        L, B, m, g = lib(), self.B, self.m, self.g
        # drafts: trees of random tokens, their distributions flat, node 0 the token decided last
        parents = np.full((B, m), -1)
        tokens = np.zeros((B, m), int)
        for b in range(B):
            par = SH.random_parents(g, new[b])
            parents[b, :new[b]] = par
            tokens[b] = g.integers(self.V, size=m)
            tokens[b, 0] = self.pending[b]
        first = SH.ints([len(t) for t in self.texts])
        d_new, d_par = SH.ints(new), SH.ints(parents)
        L.kvsel_tree_masks(d_par, self.tree, pos=self.pos, first=first, new_lens=d_new)
        L.kvsel_pages_reserve(self.params(m), self.k, self.v, self.table, self.ref, self.lens, self.granted, self.ws, new_lens=d_new)
        assert self.granted.tolist() == list(new)
        pos = self.pos.cpu().numpy()
        for b in range(B):
            if new[b]:
                self.write(b, len(self.texts[b]), tokens[b, :new[b]].tolist(), pos[b, :new[b]])
        full = self.lens + d_new
        out = torch.zeros((self.layers, B, self.H * self.G, m, D), dtype=torch.bfloat16, device="cuda")
        q = torch.stack([self.emb_q[x][torch.from_numpy(tokens).cuda()].transpose(1, 2).contiguous() for x in range(self.layers)])
        p = L.make_attn_params(h_kv=self.H, group=self.G, batch=B, n_new=m, max_len=self.cap * self.bs)
        for layer in range(self.layers):
            L.kvsel_rope(self.turn, q[layer], self.pos, new_lens=d_new)
            kv = L.make_kv_paged(self.k[layer], self.v[layer], self.table)
            L.kvsel_attend_tree(p, q[layer], kv, full, self.tree, out[layer], self.ws, new_lens=d_new)
        target = torch.softmax(out.float().mean((0, 2)) @ self.head.T, -1).contiguous()        # [B][m][V]
        draft = torch.full_like(target, 1.0 / self.V)
        u = torch.from_numpy(g.random((B, m)).astype(np.float32)).cuda()
        L.kvsel_verify(L.make_verify_params(batch=B, n_new=m, vocab=self.V), SH.ints(tokens), d_par, target, self.path, self.counts,
                       self.next, self.ws, draft=draft, u=u, new_lens=d_new)
        L.kvsel_pages_accept(self.params(m), self.k, self.v, self.table, full, self.path, self.counts, self.lens, self.ws, new_lens=d_new)
        L.kvsel_pages_trim(self.params(m), self.table, self.ref, self.lens, self.ws)
        assert CH.status(self.ws) == 0

        # every call against the oracle, from the same inputs
        got = CH.to_f64(out)
        accepted = []
        for b in range(B):
            n, mb = len(self.texts[b]), new[b]
            see = SO.ancestors(parents[b, :mb].tolist())
            assert pos[b, :mb].tolist() == (n + see.sum(axis=1) - 1).tolist()
            nodes, token = SO.verify(tokens[b, :mb].tolist(), parents[b].tolist(), target[b].cpu().numpy(), draft[b].cpu().numpy(),
                                     u[b].cpu().numpy(), "sampled")
            accepted.append(nodes)
            assert self.path[b].tolist() == nodes + [-1] * (m - len(nodes)) and int(self.counts[b]) == len(nodes)
            assert int(self.next[b]) == token
            # the tree's rows as they were before the accepted ones moved
            for layer in range(self.layers):
                seq = self.texts[b] + tokens[b, :mb].tolist()
                where = list(range(n)) + pos[b, :mb].tolist()
                k = CH.to_f64(self.turned(self.emb_k[layer][None, seq].transpose(1, 2).contiguous(), np.asarray(where)))[0]
                v = CH.to_f64(self.emb_v[layer][seq]).transpose(1, 0, 2)
                qq = CH.to_f64(q[layer, b]).reshape(self.H, self.G, m, D)
                for h in range(self.H):
                    o = SO.attend_seen(qq[h][:, :mb], k[h], v[h], SO.tree_visible(len(seq), see, 0, 0))
                    e = (D + 4) * 2.0 ** -23 * o["abs_logit"] + 2.0 ** -14          # (as in the tests of the attention)
                    tol = (2 * e[..., None] + 2.0 ** -8) * o["mean_abs"] + 2.0 ** -8 * np.abs(o["out"]) + 1e-30
                    err = np.abs(got[layer, b].reshape(self.H, self.G, m, D)[h][:, :mb] - o["out"])
                    assert np.all(err <= tol), (b, layer, h, float((err / tol).max()))
            self.texts[b] += tokens[b, nodes].tolist()
            if mb:
                self.pending[b] = token
        return accepted

    def check(self):
        """The cache holds each request's text, row by row, and no page is lost or counted wrongly."""
        table, ref = self.table.cpu().numpy(), self.ref.cpu().numpy()
        assert self.lens.tolist() == [len(t) for t in self.texts]
        uses = np.zeros_like(ref)
        for b, text in enumerate(self.texts):
            used = -(-len(text) // self.bs)
            assert (table[b, :used] >= 0).all() and (table[b, used:] == -1).all()
            np.add.at(uses, table[b, :used], 1)
            k = self.turned(self.emb_k[:, text].transpose(1, 2).contiguous(), np.arange(len(text)))
            v = self.emb_v[:, text].transpose(1, 2)
            for pool, want in ((self.k, k), (self.v, v)):
                rows = pool[:, table[b, :used]].reshape(self.layers, -1, self.H, D)[:, :len(text)].transpose(1, 2)
                assert bool((rows == want).all()), b
        assert np.array_equal(uses, ref)


@pytest.mark.parametrize("B,m,prompt", [(3, 9, 37), (2, 33, 5), (5, 4, 64)])
def test_drafted_tokens_over_shared_pages(B, m, prompt):
    loop = Loop(B, m, prompt, seed=m)
    loop.pending = loop.g.integers(loop.V, size=B).tolist()
    grown = 0
    for step in range(8):
        new = [m] * B if step % 2 else [int(loop.g.integers(0, m + 1)) for _ in range(B)]
        nodes = loop.step(new)
        loop.check()
        grown += sum(len(x) > 1 for x in nodes)
    assert grown > 0                                  # (some drafted token was accepted)


def test_a_selection_stays_and_goes_on():
    """select, kept rows in place, pages behind them freed, then eviction, new rows and attention with weights."""
    import torch

    L = lib()
    B, H, G, bs, lens = 2, 2, 4, 16, [500, 333]
    g = CH.rng(5)
    p = L.make_params(h_kv=H, group=1, n_ctx=max(lens), window=32, n_ctx_per_req=lens, n_sink=4, n_recent=16, budget_ratio=0.3)
    n_scores, n_kept, n_seg = L.kvsel_output_size(p)
    scores = np.exp(g.standard_normal(n_scores)).astype(np.float32)
    nb = -(-max(lens) // bs)
    table = np.full((B, nb), -1, np.int32)
    ids = list(g.permutation(B * nb + 4))
    for b, n in enumerate(lens):
        for i in range(-(-n // bs)):
            table[b, i] = ids.pop()
    ref = np.bincount(table[table >= 0], minlength=B * nb + 4)
    k, v = (CH.bf16(g.standard_normal((B * nb + 4, bs, H, D))) for _ in range(2))
    kd, vd, td, rd = CH.to_gpu_bf16(k), CH.to_gpu_bf16(v), SH.ints(table), SH.ints(ref)
    kv = L.make_kv_paged(kd, vd, td)
    idx, counts = SH.ints(np.zeros(n_kept)), SH.ints(np.zeros(n_seg))
    offsets = torch.zeros(n_seg, dtype=torch.int64, device="cuda")
    cap = nb * bs
    d = dict(lens=SH.ints(np.zeros((B, H))), seen=SH.ints(np.zeros((B, H))), pos=SH.ints(np.zeros((B, H, cap))),
             acc=torch.zeros((B, H, cap), device="cuda"))
    sd = torch.from_numpy(scores).cuda()
    ws = CH.workspace(1 << 24)
    L.kvsel_select(p, sd, None, idx, counts, offsets, ws)
    L.kvsel_compact_in_place(p, kv, idx, counts, offsets, d["lens"], d["seen"], d["pos"], ws, scores=sd, acc=d["acc"])
    pp = L.make_pages_params(batch=B, max_blocks=nb, num_blocks=len(ref), block_size=bs, h_kv=H, n_new=2, lens_per_head=True)
    L.kvsel_pages_trim(pp, td, rd, d["lens"], ws)
    assert CH.status(ws) == 0
    # the state here
    idx, counts = idx.cpu().numpy(), counts.cpu().numpy()
    rows_k, rows_v, pos, acc = {}, {}, {}, {}
    at = s = 0
    for b, n in enumerate(lens):
        kk, vv = (x[table[b, :-(-n // bs)]].reshape(-1, H, D)[:n] for x in (k, v))
        for h in range(H):
            where = SO.keep_rows(n, idx[s:s + counts[b * H + h]].tolist())
            s += counts[b * H + h]
            rows_k[b, h], rows_v[b, h], pos[b, h] = kk[where, h], vv[where, h], np.array(where)
            acc[b, h] = scores[at:at + n][where].astype(np.float64)
            at += n
    used = [-(-max(len(pos[b, h]) for h in range(H)) // bs) for b in range(B)]
    t2 = td.cpu().numpy()
    assert all((t2[b, :used[b]] == table[b, :used[b]]).all() and (t2[b, used[b]:] == -1).all() for b in range(B))
    assert np.array_equal(rd.cpu().numpy(), np.bincount(t2[t2 >= 0], minlength=len(ref)))
    seen, budget, m = list(lens), 120, 2
    pe = L.make_evict_params(h_kv=H, batch=B, capacity=cap, budget=budget, n_new=m, n_sink=4, n_recent=16)
    pa = L.make_attn_params(h_kv=H, group=G, batch=B, n_new=m, max_len=cap, lens_per_head=True, acc_stride=cap)
    granted = SH.ints(np.zeros(B))
    for step in range(4):
        kn, vn, qn = (CH.bf16(g.standard_normal(x)) for x in ((B, H, m, D), (B, H, m, D), (B, H * G, m, D)))
        out = CH.to_gpu_bf16(np.zeros((B, H * G, m, D)))
        L.kvsel_pages_reserve(pp, kd, vd, td, rd, d["lens"], granted, ws)
        L.kvsel_evict_append(pe, kv, d["lens"], d["seen"], d["pos"], d["acc"], CH.to_gpu_bf16(kn), CH.to_gpu_bf16(vn), ws)
        L.kvsel_attend(pa, CH.to_gpu_bf16(qn), kv, d["lens"], out, ws, acc=d["acc"])
        L.kvsel_pages_trim(pp, td, rd, d["lens"], ws)
        assert CH.status(ws) == 0 and granted.tolist() == [m] * B
        got, dp, da = CH.to_f64(out).reshape(B, H, G, m, D), d["pos"].cpu().numpy(), d["acc"].cpu().numpy()
        for b in range(B):
            for h in range(H):
                a32 = acc[b, h].astype(np.float32)
                order = CO.evict_segment(pos[b, h], a32, seen[b], m, budget=budget, n_sink=4, n_recent=16)
                rows_k[b, h] = np.concatenate([rows_k[b, h][order], kn[b, h]])
                rows_v[b, h] = np.concatenate([rows_v[b, h][order], vn[b, h]])
                pos[b, h] = np.concatenate([pos[b, h][order], seen[b] + np.arange(m)])
                n = len(pos[b, h])
                assert int(d["lens"][b, h]) == n and np.array_equal(dp[b, h, :n], pos[b, h])
                o = CO.attend_segment(qn.reshape(B, H, G, m, D)[b, h], rows_k[b, h], rows_v[b, h])
                tol = CH.token_tolerance(o, n)
                assert np.all(np.abs(got[b, h] - o["out"]) <= tol)
                acc[b, h] = da[b, h, :n].astype(np.float64)      # (its rounding decides the next eviction)
            seen[b] += m
    assert int(rd.sum()) == int((td >= 0).sum())


def test_keys_before_their_rotation():
    # cached keys turned back: what the anchors' projection takes
    L = lib()
    g = CH.rng(1)
    B, H, n = 1, 2, 300
    x, pos = CH.bf16(g.standard_normal((B, H, n, D))), np.arange(n)
    tables = {d: L.kvsel_rope_table(theta=500000.0, direction=d) for d in ("forward", "inverse")}
    k = CH.to_gpu_bf16(x)
    L.kvsel_rope(tables["forward"], k, SH.ints(pos))
    back = CH.to_gpu_bf16(np.zeros((B, H, n, D)))
    L.kvsel_rope_cache(tables["inverse"], L.make_kv_contiguous(k, k), SH.ints([n]), None, out=back, batch=B, h_kv=H, max_len=n)
    # two roundings of values no larger than the pair, 2^-8 each
    assert np.all(np.abs(CH.to_f64(back) - x) <= 2.1 * 2.0 ** -8 * (np.abs(x) + np.abs(np.roll(x, 64, -1))))
    assert L.make_kv_contiguous(back, back).stride_tok == D
