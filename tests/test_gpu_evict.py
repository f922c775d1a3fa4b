"""kvsel_evict_append against the oracle (bit-exact), and the loop it serves: evict, append,
attend with running weights, over many steps."""
import numpy as np
import pytest

from oracle import cache_oracle as CO
from tests import cache_harness as CH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    from kv_cache_eviction_window_gb300 import binding

    binding.load()
    yield


class Cache:
    """Slot caches on the device with a copy of their content here."""

    def __init__(self, *, B=1, H=2, capacity=64, lens=64, m=1, layout="contiguous", block=16, seed=0, ties=False):
        import torch

        from kv_cache_eviction_window_gb300 import binding as L

        g = CH.rng(seed)
        self.B, self.H, self.cap, self.m, self.layout, self.block = B, H, capacity, m, layout, block
        self.lens = np.broadcast_to(np.asarray(lens), (B, H)).astype(np.int32).copy()
        self.seen = (self.lens * 3 + 5).astype(np.int32)
        self.pos = np.zeros((B, H, capacity), np.int32)
        for b in range(B):
            for h in range(H):
                n = self.lens[b, h]
                self.pos[b, h, :n] = g.permutation(self.seen[b, h])[:n]
                if n:
                    # the most recent token is there, the first one too
                    self.pos[b, h, g.integers(n)] = self.seen[b, h] - 1
        self.acc = np.exp(1.5 * g.standard_normal((B, H, capacity))).astype(np.float32)
        if ties:
            self.acc = np.round(self.acc).astype(np.float32)
        self.k = CH.bf16(g.standard_normal((B, H, capacity, CH.D)))
        self.v = CH.bf16(g.standard_normal((B, H, capacity, CH.D)))
        self.dev = {x: torch.from_numpy(getattr(self, x)).cuda() for x in ("lens", "seen", "pos", "acc")}
        if layout == "paged":
            nb = -(-capacity // block)
            table = g.permutation(B * nb).reshape(B, nb).astype(np.int32)
            self.table = table
            pools = []
            for x in (self.k, self.v):
                pool = np.zeros((B * nb, block, H, CH.D))
                rows = np.zeros((B, nb * block, H, CH.D))
                rows[:, :capacity] = x.transpose(0, 2, 1, 3)
                pool[table] = rows.reshape(B, nb, block, H, CH.D)
                pools.append(CH.to_gpu_bf16(pool))
            self.kt, self.vt = pools
            self.tt = torch.from_numpy(table).cuda()
            self.kv = L.make_kv_paged(self.kt, self.vt, self.tt)
        else:
            self.kt, self.vt = CH.to_gpu_bf16(self.k), CH.to_gpu_bf16(self.v)
            self.kv = L.make_kv_contiguous(self.kt, self.vt)

    def rows(self):
        if self.layout != "paged":
            return CH.to_f64(self.kt), CH.to_f64(self.vt)
        got = []
        for x in (self.kt, self.vt):
            r = CH.to_f64(x)[self.table].reshape(self.B, -1, self.H, CH.D)[:, :self.cap]
            got.append(r.transpose(0, 2, 1, 3))
        return got

    def step(self, g, *, budget, n_sink, n_recent, new=None, ws=None, strided=False):
        """One call, and the same on the copy."""
        import torch

        from kv_cache_eviction_window_gb300 import binding as L

        m = self.m
        kn, vn = (CH.bf16(g.standard_normal((self.B, self.H, m, CH.D))) for _ in range(2))
        p = L.make_evict_params(h_kv=self.H, batch=self.B, capacity=self.cap, budget=budget, n_new=m, n_sink=n_sink,
                                n_recent=n_recent)
        if strided:   # [request][token][head] slices of a projection's output
            wide = [CH.to_gpu_bf16(np.full((self.B, m, 3 * self.H, CH.D), np.nan)) for _ in range(2)]
            kd, vd = (x[:, :, self.H:2 * self.H].permute(0, 2, 1, 3) for x in wide)
            kd.copy_(CH.to_gpu_bf16(kn))
            vd.copy_(CH.to_gpu_bf16(vn))
            p.new_stride_req, p.new_stride_head, p.new_stride_tok = kd.stride()[:3]
        else:
            kd, vd = (CH.to_gpu_bf16(x) if m else None for x in (kn, vn))
        ws = ws if ws is not None else CH.workspace(L.kvsel_evict_append_workspace_size(p))
        nl = None if new is None else torch.from_numpy(np.asarray(new, np.int32)).cuda()
        d = self.dev
        L.kvsel_evict_append(p, self.kv, d["lens"], d["seen"], d["pos"], d["acc"], kd, vd, ws, new_lens=nl)
        for b in range(self.B):
            mb = m if new is None else int(new[b])
            for h in range(self.H):
                n, seen = int(self.lens[b, h]), int(self.seen[b, h])
                order = CO.evict_segment(self.pos[b, h, :n], self.acc[b, h, :n], seen, mb, budget=budget, n_sink=n_sink,
                                         n_recent=n_recent)
                keep = len(order)
                for x in (self.pos, self.acc, self.k, self.v):
                    x[b, h, :keep] = x[b, h, order]
                self.pos[b, h, keep:keep + mb] = seen + np.arange(mb)
                self.acc[b, h, keep:keep + mb] = 0
                self.k[b, h, keep:keep + mb] = kn[b, h, :mb]
                self.v[b, h, keep:keep + mb] = vn[b, h, :mb]
                self.lens[b, h] = keep + mb
                self.seen[b, h] = seen + mb
        return ws

    def check(self):
        for x in ("lens", "seen", "pos", "acc"):
            np.testing.assert_array_equal(self.dev[x].cpu().numpy(), getattr(self, x), err_msg=x)
        k, v = self.rows()
        np.testing.assert_array_equal(k, self.k)
        np.testing.assert_array_equal(v, self.v)


@pytest.mark.parametrize("layout,block", [("contiguous", 0), ("paged", 8), ("paged", 64)])
@pytest.mark.parametrize("n,m,budget,n_sink,n_recent", [
    (64, 1, 64, 4, 16), (64, 0, 20, 4, 8), (64, 0, 64, 0, 0), (1, 1, 1, 0, 1), (1, 1, 1, 0, 0), (0, 1, 5, 0, 0),
    (0, 0, 5, 0, 0), (70, 30, 70, 4, 30), (70, 70, 70, 0, 3), (1500, 1, 1500, 4, 100), (1500, 700, 1400, 1, 700),
    (1500, 3, 1000, 4, 996), (2600, 0, 1, 1, 0), (2600, 2, 2, 0, 2), (5000, 513, 4100, 64, 200)])
def test_one_call(layout, block, n, m, budget, n_sink, n_recent):
    c = Cache(B=2, H=2, capacity=max(n, budget), lens=n, m=m, layout=layout, block=block, seed=n + m)
    ws = c.step(CH.rng(1), budget=budget, n_sink=n_sink, n_recent=n_recent)
    assert CH.status(ws) == 0
    c.check()


@pytest.mark.parametrize("m", [1, 2, 5, 40])
def test_many_calls_in_a_row(m):
    g = CH.rng(m)
    c = Cache(B=2, H=3, capacity=150, lens=g.integers(0, 150, (2, 3)), m=m, seed=m, ties=True)
    ws = None
    for i in range(40):
        new = g.integers(0, m + 1, 2) if i % 3 == 0 else None
        ws = c.step(g, budget=150 - i % 5, n_sink=2, n_recent=m + i % 4, new=new, ws=ws, strided=i % 2 == 1)
    assert CH.status(ws) == 0
    c.check()


def test_weights_of_every_kind():
    import torch

    # NaN last, then -inf; zeros of either sign equal; +inf first; everything tied
    vals = np.array([np.nan, -np.inf, -1.5, -0.0, 0.0, 1e-42, 3.4e38, np.inf], np.float32)
    for seed, pick in ((1, lambda g, s: vals[g.integers(0, 8, s)]), (2, lambda g, s: np.zeros(s, np.float32)),
                       (3, lambda g, s: np.full(s, np.nan, np.float32))):
        c = Cache(capacity=300, lens=300, m=3, seed=seed)
        c.acc = pick(CH.rng(seed), c.acc.shape)
        c.dev["acc"] = torch.from_numpy(c.acc.copy()).cuda()
        for n_recent in (3, 100):
            ws = c.step(CH.rng(9), budget=250, n_sink=1, n_recent=n_recent)
            assert CH.status(ws) == 0
            c.check()


def test_bad_lengths_and_blocks_are_reported():
    from kv_cache_eviction_window_gb300 import binding as L

    c = Cache(capacity=64, lens=64, m=1, layout="paged", block=8)
    c.dev["lens"].fill_(200)                      # clamped to the capacity
    ws = c.step(CH.rng(1), budget=60, n_sink=1, n_recent=2)
    assert CH.status(ws) == -7
    c.check()
    # a block out of range: its rows are neither read nor written
    c = Cache(capacity=64, lens=64, m=4, layout="paged", block=8)
    before = c.kt.clone()
    c.tt.fill_(-1)
    ws = c.step(CH.rng(1), budget=60, n_sink=1, n_recent=4)
    assert CH.status(ws) == -7
    assert (before == c.kt).all()
    assert L.kvsel_get_device_status(ws) == 0


@pytest.mark.parametrize("n,m", [(60000, 5), (60000, 0), (49152, 300), (49153, 300)])
def test_caches_beyond_shared_memory(n, m):
    c = Cache(H=1, capacity=n, lens=n, m=m, seed=n, ties=True)
    ws = c.step(CH.rng(1), budget=n - 1000, n_sink=4, n_recent=300)
    assert CH.status(ws) == 0
    c.check()


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("B,H,n,m,budget", [
    (1, 1, 60000, 5, 59980), (1, 2, 900, 40, 890), (2, 2, 300, 64, 300), (2, 2, 300, 65, 300), (3, 1, 70, 0, 10),
    (20, 8, 120, 30, 110), (19, 8, 90, 6, 90)])
def test_few_rows_to_move(B, H, n, m, budget, ties):
    # by the block that selects them, or by a second launch; caches that are not full among them
    c = Cache(B=B, H=H, capacity=n, lens=n - np.arange(B * H).reshape(B, H) % 7, m=m, seed=n + m, ties=ties)
    g, ws = CH.rng(1), None
    for _ in range(2):
        ws = c.step(g, budget=budget, n_sink=2, n_recent=min(60, budget // 3), new=m - np.arange(B) % (m + 1), ws=ws)
    assert CH.status(ws) == 0
    c.check()


@pytest.mark.parametrize("m", [1, 30])
def test_a_captured_call_follows_the_lengths(m):
    import torch

    from kv_cache_eviction_window_gb300 import binding as L

    c = Cache(B=2, H=2, capacity=100, lens=[[100, 40], [99, 71]], m=m, seed=m)
    g = CH.rng(1)
    kn, vn = (CH.bf16(g.standard_normal((2, 2, m, CH.D))) for _ in range(2))
    kd, vd = CH.to_gpu_bf16(kn), CH.to_gpu_bf16(vn)
    p = L.make_evict_params(h_kv=2, batch=2, capacity=100, budget=100, n_new=m, n_sink=2, n_recent=m)
    ws = CH.workspace(L.kvsel_evict_append_workspace_size(p))
    d = c.dev
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.kvsel_evict_append(p, c.kv, d["lens"], d["seen"], d["pos"], d["acc"], kd, vd, ws)
    for _ in range(3):
        graph.replay()
        for b in range(2):
            for h in range(2):
                n, seen = int(c.lens[b, h]), int(c.seen[b, h])
                order = CO.evict_segment(c.pos[b, h, :n], c.acc[b, h, :n], seen, m, budget=100, n_sink=2, n_recent=m)
                keep = len(order)
                for x in (c.pos, c.acc, c.k, c.v):
                    x[b, h, :keep] = x[b, h, order]
                c.pos[b, h, keep:keep + m] = seen + np.arange(m)
                c.acc[b, h, keep:keep + m] = 0
                c.k[b, h, keep:keep + m] = kn[b, h]
                c.v[b, h, keep:keep + m] = vn[b, h]
                c.lens[b, h], c.seen[b, h] = keep + m, seen + m
    assert CH.status(ws) == 0
    c.check()


def test_decode_loop_with_eviction():
    """A prompt is compacted, then tokens arrive one by one (and in a chunk): evict and append,
    attend with running weights.  The copy follows with the oracle; the weights that the next
    eviction ranks are the device's own."""
    import torch

    from kv_cache_eviction_window_gb300 import binding as L

    B, H, G, cap = 2, 2, 4, 200
    g = CH.rng(7)
    c = Cache(B=B, H=H, capacity=cap, lens=cap, m=1, layout="paged", block=16, seed=7)
    ws = CH.workspace(1 << 26)
    for m in (1, 1, 1, 17, 1, 1):
        c.m = m
        c.step(g, budget=cap, n_sink=2, n_recent=20, ws=ws)
        c.check()
        q = CH.bf16(g.standard_normal((B, H, G, m, CH.D)) * 1.5)
        p = L.make_attn_params(h_kv=H, group=G, batch=B, n_new=m, max_len=cap, lens_per_head=True, acc_stride=cap)
        assert L.kvsel_attend_workspace_size(p, True) <= ws.numel()
        out = torch.empty((B, H * G, m, CH.D), dtype=torch.bfloat16, device="cuda")
        L.kvsel_attend(p, CH.to_gpu_bf16(q.reshape(B, H * G, m, CH.D)), c.kv, c.dev["lens"], out, ws, acc=c.dev["acc"])
        assert CH.status(ws) == 0
        got, acc = CH.to_f64(out).reshape(B, H, G, m, CH.D), c.dev["acc"].cpu().numpy()
        for b in range(B):
            for h in range(H):
                n = c.lens[b, h]
                o = CO.attend_segment(q[b, h], c.k[b, h, :n], c.v[b, h, :n])
                e = 132 * 2.0 ** -23 * o["abs_logit"] + 2.0 ** -14
                tol = (2 * e[..., None] + 2.0 ** -8) * o["mean_abs"] + 2.0 ** -8 * np.abs(o["out"])
                assert np.all(np.abs(got[b, h] - o["out"]) <= tol)
                want = c.acc[b, h, :n] + o["weight"]
                et = (2 * e.max() + (G * m + 2) * 2.0 ** -23) * o["weight"] + 2.0 ** -23 * np.abs(want)
                assert np.all(np.abs(acc[b, h, :n] - want) <= et)
        c.acc = acc.copy()
