"""Helpers of the tests of a step of drafted tokens.  Importing this module does not need a GPU."""
import numpy as np

from oracle import step_oracle as SO
from tests import cache_harness as CH

D = CH.D


def random_parents(g, m, kind="tree"):
    if kind == "chain":
        return [t - 1 for t in range(m)]
    if kind == "star":
        return [-1] + [0] * (m - 1)
    return [-1] + [t - 1 if g.random() < 0.4 else int(g.integers(t)) for t in range(1, m)] if m else []


class TreeCase(CH.Case):
    """One call of kvsel_attend_tree: `masks` [B] of [m][m] bool, or trees of random parents."""

    def __init__(self, *, masks=None, kind="tree", **kw):
        super().__init__(**kw)
        self.masks = masks or [SO.ancestors(random_parents(self.g, int(x), kind)) for x in self.new]

    def seen(self, b, h):
        return SO.tree_visible(int(self.lens[b][h]), self.masks[b], self.window, self.n_sink)

    def seen_rows(self, b, h):
        # what must be finite: rows that a token at row n - m sees, and the tree's
        n, m = int(self.lens[b][h]), int(self.new[b])
        if m == 0:
            return np.zeros(n, bool)
        root = SO.tree_visible(n, np.eye(m, dtype=bool)[:, :m], self.window, self.n_sink)[0] if n else np.zeros(0, bool)
        root[max(0, n - m):] = True
        return root

    def oracle(self):
        return [[SO.attend_seen(self.q[b, h, :, :self.new[b]], np.where(self.seen_rows(b, h)[:, None], self.k[b][h], 0.0),
                                np.where(self.seen_rows(b, h)[:, None], self.v[b][h], 0.0), self.seen(b, h), self.scale or None)
                 for h in range(self.H)] for b in range(self.B)]

    def upload(self):
        import torch

        super().upload()
        W = -(-self.m // 32)
        tree = np.full((self.B, self.m, W), 0xA5A5A5A5, np.uint32)   # masks behind a request's nodes: anything
        for b in range(self.B):
            m = int(self.new[b])
            full = SO.words(self.masks[b], self.m)
            # bits of rows behind the request's nodes: anything
            for t in range(m):
                row = sum(int(x) << 32 * w for w, x in enumerate(full[t])) | ((0x5A5A5A5A5A << m) & ((1 << 32 * W) - 1))
                tree[b, t] = [row >> 32 * w & 0xFFFFFFFF for w in range(W)]
        self.t["tree"] = torch.from_numpy(tree.view(np.int32)).cuda()
        return self

    def call(self, ws=None, stream=None, lse=True):
        from kv_cache_eviction_window_gb300 import binding as L

        p = L.make_attn_params(**{**self.params, "acc_stride": 0})
        if ws is None:
            ws = CH.workspace(L.kvsel_attend_tree_workspace_size(p))
        t = self.t
        L.kvsel_attend_tree(p, t["q"], t["kv"], t["lens"], t["tree"], t["out"], ws, new_lens=t["new_lens"], offsets=self.offsets,
                            lse=t["lse"] if lse else None, stream=stream)
        return ws


def run_tree(**kw):
    c = TreeCase(**kw).upload()
    ws = c.call()
    assert CH.status(ws) == 0
    c.check()
    return c


def ints(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def probabilities(g, shape, sharp=2.0, zeros=0.0):
    """Rows of float32 probabilities, a share of them zero."""
    x = np.exp(sharp * g.standard_normal(shape))
    if zeros:
        x *= g.random(shape) >= zeros
        x[..., 0] += 1e-3
    return (x / x.sum(axis=-1, keepdims=True)).astype(np.float32)


class VerifyCase:
    """One call of kvsel_verify with trees whose nodes are drafted as the mode says."""

    def __init__(self, *, B=2, m=8, V=100, mode="sampled", dtype="fp32", kind="tree", new=None, seed=0, near=0.6, zeros=0.0, sharp=2.0):
        g = CH.rng(seed)
        self.B, self.m, self.V, self.mode, self.dtype, self.g = B, m, V, mode, dtype, g
        self.new = np.full(B, m) if new is None else np.asarray(new)
        self.new_given = new is not None
        logits = sharp * g.standard_normal((B, m, V))
        guess = logits + near * g.standard_normal((B, m, V))
        soft = lambda x: np.exp(x - x.max(-1, keepdims=True)) / np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)   # noqa: E731
        p, q = soft(logits), soft(guess)
        if zeros:
            p, q = p * (g.random(p.shape) >= zeros), q * (g.random(q.shape) >= zeros)
            q[..., 0] += 1e-6
            p, q = p / np.maximum(p.sum(-1, keepdims=True), 1e-30), q / q.sum(-1, keepdims=True)
        self.p = logits if mode == "greedy" else p
        self.q = q if mode == "sampled" else None
        rnd = CH.bf16 if dtype == "bf16" else (lambda x: x.astype(np.float32).astype(np.float64))
        self.p = rnd(self.p)
        self.q = None if self.q is None else rnd(self.q)
        self.parents = np.full((B, m), -1)
        self.tokens = np.zeros((B, m), int)
        for b in range(B):
            par = random_parents(g, int(self.new[b]), kind)
            self.parents[b, :len(par)] = par
            for t in range(1, len(par)):
                c = par[t]
                if mode == "sampled":
                    w = self.q[b, c]
                    self.tokens[b, t] = min(int(np.searchsorted(np.cumsum(w), g.random() * w.sum(), side="right")), V - 1)
                else:
                    rank = sum(x == c for x in par[:t])
                    self.tokens[b, t] = np.argsort(-guess[b, c], kind="stable")[min(rank, V - 1)]
        self.u = g.random((B, m)).astype(np.float32)

    def oracle(self):
        return [SO.verify(self.tokens[b, :self.new[b]].tolist(), self.parents[b].tolist(), self.p[b], None if self.q is None else self.q[b],
                          self.u[b], self.mode) for b in range(self.B)]

    def upload(self, pad=0, lead=0):
        """pad: elements between nodes' rows; lead: elements before the first."""
        import torch

        def put(x):
            if x is None:
                return None
            wide = np.full((self.B, self.m, self.V + pad), np.nan)
            wide[..., :self.V] = x
            flat = np.concatenate([np.full(lead, np.nan), wide.reshape(-1)])
            t = CH.to_gpu_bf16(flat) if self.dtype == "bf16" else torch.from_numpy(flat.astype(np.float32)).cuda()
            return t[lead:].view(self.B, self.m, self.V + pad)[..., :self.V]

        self.pad = pad
        self.t = dict(tokens=ints(self.tokens), parents=ints(self.parents), target=put(self.p), draft=put(self.q),
                      u=torch.from_numpy(self.u).cuda(), new_lens=ints(self.new) if self.new_given else None,
                      path=ints(np.full((self.B, self.m), 7)), counts=ints(np.full(self.B, 7)), next=ints(np.full(self.B, 7)))
        return self

    def call(self, ws=None, stream=None):
        from kv_cache_eviction_window_gb300 import binding as L

        V = self.V + self.pad
        p = L.make_verify_params(batch=self.B, n_new=self.m, vocab=self.V, mode=self.mode, dtype=self.dtype,
                                 stride_req=self.m * V if self.pad else 0, stride_node=V if self.pad else 0)
        if ws is None:
            ws = CH.workspace(max(256 + 65536, L.kvsel_verify_workspace_size(p)))
        t = self.t
        L.kvsel_verify(p, t["tokens"], t["parents"], t["target"], t["path"], t["counts"], t["next"], ws, draft=t["draft"],
                       u=None if self.mode == "greedy" else t["u"], new_lens=t["new_lens"], stream=stream)
        return ws

    def check(self, want=None):
        want = want or self.oracle()
        path, counts, nxt = (self.t[x].cpu().numpy() for x in ("path", "counts", "next"))
        for b, (nodes, token) in enumerate(want):
            assert counts[b] == len(nodes), (b, counts[b], nodes)
            assert path[b].tolist() == nodes + [-1] * (self.m - len(nodes)), b
            assert nxt[b] == token, (b, nxt[b], token)


class PageCase:
    """Tables with random pages, pools of random bits, and the same state in the oracle."""

    def __init__(self, *, B=4, H=2, L=2, bs=16, rows=(40,), cap=8, spare=20, share=None, seed=0, per_head=False):
        g = CH.rng(seed)
        self.B, self.H, self.L, self.bs, self.cap, self.per_head, self.g = B, H, L, bs, cap, per_head, g
        self.lens = np.resize(np.asarray(rows), (B, H) if per_head else (B,)).astype(np.int32)
        top = self.lens.reshape(B, -1).max(axis=1)
        total = int(sum(-(-n // bs) for n in top)) + spare
        ids = list(g.permutation(total))
        table, ref = np.full((B, cap), -1, np.int32), np.zeros(total, np.int32)
        for b in range(B):
            used, of = -(-int(top[b]) // bs), None if share is None else share[b]
            for i in range(used):
                table[b, i] = table[of, i] if of is not None and table[of, i] >= 0 else ids.pop()
                ref[table[b, i]] += 1
        k, v = (g.integers(0, 65536, (L, total, bs, H, D)).astype(np.uint16) for _ in range(2))
        self.o = SO.Pages(table, ref, k, v)

    def params(self, n_new):
        from kv_cache_eviction_window_gb300 import binding as L

        return L.make_pages_params(batch=self.B, max_blocks=self.cap, num_blocks=len(self.o.ref), block_size=self.bs, h_kv=self.H,
                                   layers=self.L, n_new=n_new, lens_per_head=self.per_head)

    def upload(self):
        import torch

        self.table, self.other, self.ref, self.d_lens = ints(self.o.table), ints(self.o.table * 0 + 77), ints(self.o.ref), ints(self.lens)
        self.k, self.v = (torch.from_numpy(x.view(np.int16)).cuda() for x in (self.o.k, self.o.v))
        from kv_cache_eviction_window_gb300 import binding as L

        self.ws = CH.workspace(L.kvsel_pages_workspace_size(self.params(8192)))
        return self

    def check(self, table=None):
        assert np.array_equal((self.table if table is None else table).cpu().numpy(), self.o.table)
        assert np.array_equal(self.ref.cpu().numpy(), self.o.ref)
        for t, x in ((self.k, self.o.k), (self.v, self.o.v)):
            assert np.array_equal(t.cpu().numpy().view(np.uint16), x)
