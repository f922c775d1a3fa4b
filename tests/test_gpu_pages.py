"""kvsel_pages_* and kvsel_compact_in_place, bit for bit against the oracle: forks, reservations with copies of
shared pages, freed pages, accepted rows in every layer, kept rows in place, and the loops that they make."""
import numpy as np
import pytest

from oracle import step_oracle as SO
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


def reserve(c, new, n_new=None):
    p, granted = c.params(n_new or max(max(new), 1)), SH.ints(np.full(c.B, 7))
    lib().kvsel_pages_reserve(p, c.k, c.v, c.table, c.ref, c.d_lens, granted, c.ws, new_lens=SH.ints(new))
    want = c.o.reserve(c.lens, new)
    st = CH.status(c.ws)
    assert np.array_equal(granted.cpu().numpy(), want), (granted, want)
    return want, st


@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("new", [[0, 0, 0], [1, 1, 1], [1, 0, 40], [9, 64, 5], [200, 7, 130]])
def test_reserve(bs, new):
    c = SH.PageCase(B=3, H=2, L=3, bs=bs, rows=[40, 16, 0], cap=40, spare=70, seed=bs).upload()
    assert reserve(c, new)[1] == 0
    c.check()
    assert reserve(c, new)[1] == 0      # what is reserved already stays
    c.check()


@pytest.mark.parametrize("share,rows", [([None, 0, 0, 0], [21, 21, 21, 21]), ([None, None, 1, 1], [16, 33, 33, 33]),
                                        ([None, 0, None, 2], [5, 5, 64, 64]), ([None, 0, 0, None], [31, 16, 5, 1])])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [0, 3, 0, 2], [20, 1, 17, 40]])
def test_shared_pages_are_copied(share, rows, new):
    c = SH.PageCase(B=4, H=3, L=4, rows=rows, cap=12, spare=30, share=share, seed=len(rows)).upload()
    assert reserve(c, new)[1] == 0
    c.check()


@pytest.mark.parametrize("spare", range(9))
def test_when_pages_run_out(spare):
    c = SH.PageCase(B=5, rows=[16, 21, 21, 16, 21], share=[None, None, 1, None, 1], cap=8, spare=spare, seed=spare).upload()
    reserve(c, [17, 1, 1, 16, 0])
    c.check()


@pytest.mark.parametrize("n_new", [64, 8192])
@pytest.mark.parametrize("spare", [0, 1, 2, 3])
def test_a_page_is_taken_over_only_from_those_that_leave_it(n_new, spare):
    # request 0 has more rows on the shared page than request 1: left with it, 1 would write over them
    def case(**kw):                                   # of the free pages `spare` are left (those not needed twice are free, too)
        c = SH.PageCase(cap=8, seed=spare, **kw)
        c.o.ref[np.flatnonzero(c.o.ref == 0)[spare:]] = 1
        return c.upload()

    c = case(B=4, rows=[23, 18, 23, 7], share=[None, 0, 0, None])
    granted, st = reserve(c, [3, 2, 0, 1], n_new=n_new)
    assert st == 0 and granted.tolist() == [3 * (spare > 0), 2 * (spare > 1), 0, 1]
    c.check()
    c = case(B=2, rows=[23, 18], share=[None, 0])
    granted, st = reserve(c, [3, 2], n_new=n_new)
    assert st == 0 and granted.tolist() == ([3, 2] if spare else [0, 0])
    c.check()


@pytest.mark.parametrize("n_new", [64, 8192])
def test_a_page_of_a_request_that_is_refused_stays_its_own(n_new):
    c = SH.PageCase(B=2, rows=[23, 18], share=[None, 0], cap=8, spare=5, seed=3).upload()
    page = int(c.table[0, 1])
    c.table[0, 2] = 10 ** 6
    granted = SH.ints([7, 7])
    lib().kvsel_pages_reserve(c.params(n_new), c.k, c.v, c.table, c.ref, c.d_lens, granted, c.ws, new_lens=SH.ints([20, 2]))
    assert CH.status(c.ws) == -7 and granted.tolist() == [0, 2]
    to = int(np.flatnonzero(c.o.ref == 0)[0])
    assert c.table[:, 1].tolist() == [page, to] and c.ref[page] == 1 and c.ref[to] == 1
    want = c.o.k.copy()
    want[:, to, :2] = want[:, page, :2]               # (its rows 16 and 17)
    assert np.array_equal(c.k.cpu().numpy().view(np.uint16), want)


def test_heads_of_different_lengths():
    rows = [[5, 20, 33], [16, 16, 0], [0, 0, 0], [64, 1, 30]]
    for share in (None, [None, None, None, 0]):
        c = SH.PageCase(B=4, H=3, L=2, rows=rows, per_head=True, cap=10, spare=30, share=share, seed=2).upload()
        assert reserve(c, [30, 17, 1, 4], n_new=64)[1] == 0
        c.check()


def test_requests_that_cannot_be_served():
    # beyond the table's row; a length or count out of range; the others are served
    c = SH.PageCase(B=4, rows=[100, 20, 20, 20], cap=8, spare=30, seed=1).upload()
    assert reserve(c, [40, 3, 3, 3])[1] == -7
    c.check()
    c = SH.PageCase(B=2, rows=[20, 20], cap=8, spare=30, seed=1).upload()
    granted = SH.ints([7, 7])
    c.d_lens[0] = -1
    lib().kvsel_pages_reserve(c.params(4), c.k, c.v, c.table, c.ref, c.d_lens, granted, c.ws, new_lens=SH.ints([4, 5]))
    assert CH.status(c.ws) == -7
    assert granted.tolist() == [0, 0]
    c.check()
    c.d_lens.copy_(SH.ints([20, 20]))
    c.table[0, 1] = 10 ** 6
    lib().kvsel_pages_reserve(c.params(4), c.k, c.v, c.table, c.ref, c.d_lens, granted, c.ws)
    assert CH.status(c.ws) == -7
    assert granted.tolist() == [0, 4]


@pytest.mark.parametrize("cap", [1, 7, 300, 1000])
def test_fork(cap):
    c = SH.PageCase(B=6, H=2, L=1, rows=[16 * cap, 5, 0, 16 * cap - 3, 1, 16], cap=cap, spare=3, seed=cap).upload()
    src, out = [0, 0, 3, -1, 0, 5], SH.ints(np.zeros(6))
    lib().kvsel_pages_fork(c.params(1), c.table, c.d_lens, SH.ints(src), c.other, out, c.ref, c.ws)
    assert CH.status(c.ws) == 0
    c.o.fork(src)
    c.check(c.other)
    assert out.tolist() == [int(c.lens[s]) if s >= 0 else 0 for s in src]


def test_fork_per_head_and_bad_sources():
    c = SH.PageCase(B=3, H=2, rows=[[5, 20], [16, 16], [0, 0]], per_head=True, cap=4, seed=1).upload()
    out = SH.ints(np.zeros((3, 2)))
    lib().kvsel_pages_fork(c.params(1), c.table, c.d_lens, SH.ints([1, 0, 0]), c.other, out, c.ref, c.ws)
    c.o.fork([1, 0, 0])
    assert CH.status(c.ws) == 0
    c.check(c.other)
    assert np.array_equal(out.cpu().numpy(), c.lens[[1, 0, 0]])
    c = SH.PageCase(B=3, rows=[5, 20, 33], cap=4, seed=1).upload()
    out = SH.ints(np.zeros(3))
    lib().kvsel_pages_fork(c.params(1), c.table, c.d_lens, SH.ints([3, -2, 1]), c.other, out, c.ref, c.ws)
    c.o.fork([-1, -1, 1])
    assert CH.status(c.ws) == -7
    c.check(c.other)


def test_trim():
    for per_head in (False, True):
        c = SH.PageCase(B=4, H=2, rows=[[60, 50], [33, 2], [16, 16], [0, 0]] if per_head else [60, 33, 16, 0], per_head=per_head,
                        share=[None, 0, None, None], cap=9, seed=1).upload()
        now = np.array([[17, 3], [0, 32], [16, 1], [0, 0]] if per_head else [17, 32, 0, 0], np.int32)
        lib().kvsel_pages_trim(c.params(1), c.table, c.ref, SH.ints(now), c.ws)
        assert CH.status(c.ws) == 0
        c.o.trim(now)
        c.check()
    lib().kvsel_pages_trim(c.params(1), c.table, c.ref, SH.ints(now * 0 - 1), c.ws)
    assert CH.status(c.ws) == -7
    c.check()


@pytest.mark.parametrize("m", [1, 2, 9, 40, 200])
@pytest.mark.parametrize("L", [1, 5])
def test_accept(m, L):
    c = SH.PageCase(B=5, H=2, L=L, rows=[16 * 13 + m, m, 40 + m, 5, 300], cap=40, seed=m).upload()
    new = [m, m, max(1, m // 2), min(m, 2), 0]
    paths = [sorted({0} | set(c.g.choice(x, size=c.g.integers(0, x + 1), replace=False).tolist())) if x else [] for x in new]
    paths[1] = list(range(m))
    path = np.full((5, m), -1)
    for b, x in enumerate(paths):
        path[b, :len(x)] = x
    out = SH.ints(np.zeros(5))
    lib().kvsel_pages_accept(c.params(m), c.k, c.v, c.table, c.d_lens, SH.ints(path), SH.ints([len(x) for x in paths]), out, c.ws,
                             new_lens=SH.ints(new))
    assert CH.status(c.ws) == 0
    want = c.o.accept(c.lens, new, paths)
    c.check()
    assert np.array_equal(out.cpu().numpy(), want)
    # lengths in place
    c = SH.PageCase(B=5, H=2, L=L, rows=[16 * 13 + m, m, 40 + m, 5, 300], cap=40, seed=m).upload()
    lib().kvsel_pages_accept(c.params(m), c.k, c.v, c.table, c.d_lens, SH.ints(path), SH.ints([len(x) for x in paths]), c.d_lens, c.ws,
                             new_lens=SH.ints(new))
    c.o.accept(c.lens, new, paths)
    c.check()
    assert np.array_equal(c.d_lens.cpu().numpy(), want)


def test_accept_per_head():
    c = SH.PageCase(B=2, H=3, rows=[[40, 21, 33], [9, 64, 10]], per_head=True, cap=6, seed=1).upload()
    paths, m = [[0, 3, 8], [0, 1, 5, 6]], 9
    path = np.full((2, m), -1)
    for b, x in enumerate(paths):
        path[b, :len(x)] = x
    out = SH.ints(np.zeros((2, 3)))
    lib().kvsel_pages_accept(c.params(m), c.k, c.v, c.table, c.d_lens, SH.ints(path), SH.ints([3, 4]), out, c.ws)
    assert CH.status(c.ws) == 0
    want = c.o.accept(c.lens, [m, m], paths)
    c.check()
    assert np.array_equal(out.cpu().numpy(), want)


def test_accept_records_what_is_wrong():
    c = SH.PageCase(B=2, rows=[40, 20], cap=6, seed=1).upload()
    out = SH.ints([0, 0])
    # an entry below its place, one not above the one before, one behind the tree: the rest moves
    path = [[0, 0, 5, 5, 6, 9, -1, -1, -1], [0, 2, 3, -1, -1, -1, -1, -1, -1]]
    lib().kvsel_pages_accept(c.params(9), c.k, c.v, c.table, c.d_lens, SH.ints(path), SH.ints([6, 3]), out, c.ws)
    assert CH.status(c.ws) == -7
    assert out.tolist() == [40 - 9 + 6, 20 - 9 + 3]
    o = c.o
    for b, moves in enumerate([[(5, 2), (6, 4)], [(2, 1), (3, 2)]]):
        base = int(c.lens[b]) - 9
        for x, i in moves:
            (p0, s0), (p1, s1) = divmod(base + x, 16), divmod(base + i, 16)
            for pool in (o.k, o.v):
                pool[:, o.table[b, p1], s1] = pool[:, o.table[b, p0], s0]
    c.check()


def test_a_search_with_beams():
    # 3 prompts of 3 beams: fork by what the search chose, reserve, append by hand; at the end everything is free
    B, bs = 9, 16
    c = SH.PageCase(B=B, H=2, L=2, bs=bs, rows=[30, 30, 30, 47, 47, 47, 3, 3, 3], share=[None, 0, 0, None, 3, 3, None, 6, 6], cap=8,
                    spare=25, seed=4).upload()
    a, b, la, lb = c.table, c.other, c.d_lens, SH.ints(np.zeros(B))
    granted = SH.ints(np.zeros(B))
    for step in range(40):
        src = [3 * (x // 3) + int(c.g.integers(3)) for x in range(B)]
        lib().kvsel_pages_fork(c.params(1), a, la, SH.ints(src), b, lb, c.ref, c.ws)
        c.o.fork(src)
        c.lens = c.lens[src]
        lib().kvsel_pages_reserve(c.params(1), c.k, c.v, b, c.ref, lb, granted, c.ws)
        assert np.array_equal(c.o.reserve(c.lens, [1] * B), granted.cpu().numpy())
        for x in range(B):
            page, slot = c.o.table[x, c.lens[x] // bs], c.lens[x] % bs
            c.o.k[:, page, slot] = c.o.v[:, page, slot] = step * 16 + x
            c.k[:, page, slot] = c.v[:, page, slot] = step * 16 + x
        lb += 1
        c.lens = c.lens + 1
        c.check(b)
        a, b, la, lb = b, a, lb, la
    lib().kvsel_pages_trim(c.params(1), a, c.ref, SH.ints(np.zeros(B)), c.ws)
    assert CH.status(c.ws) == 0
    assert int(c.ref.abs().sum()) == 0 and int((a + 1).abs().sum()) == 0


def test_many_pages_and_requests():
    # the scan for free pages goes far; a request of many pages beside small ones
    c = SH.PageCase(B=200, H=1, L=1, bs=8, rows=[8 * (i % 5) + i % 8 for i in range(200)], cap=700, spare=7000, seed=4).upload()
    c.o.ref[:5000] = np.maximum(c.o.ref[:5000], 1)
    c.ref.copy_(SH.ints(c.o.ref))
    new = [(i * 7) % 20 for i in range(200)]
    new[3] = 5000
    assert reserve(c, new)[1] == 0
    c.check()


def test_captured():
    import torch

    B = 4
    c = SH.PageCase(B=B, rows=[21, 21, 21, 37], share=[None, 0, 0, None], cap=8, spare=30, seed=4).upload()
    granted, out = SH.ints(np.zeros(B)), SH.ints(np.zeros(B))
    m, path, counts = 5, SH.ints([[0, 2, 3, -1, -1]] * B), SH.ints([3] * B)
    more = SH.ints(c.lens + m)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    p = c.params(m)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            lib().kvsel_pages_reserve(p, c.k, c.v, c.table, c.ref, c.d_lens, granted, c.ws)
            lib().kvsel_pages_accept(p, c.k, c.v, c.table, more, path, counts, out, c.ws)
            lib().kvsel_pages_trim(p, c.table, c.ref, out, c.ws)
    for _ in range(3):
        g.replay()
        c.o.reserve(c.lens, [m] * B)
        now = c.o.accept(c.lens + m, [m] * B, [[0, 2, 3]] * B)
        c.o.trim(now)
    assert CH.status(c.ws) == 0
    c.check()
    assert np.array_equal(out.cpu().numpy(), now)


# ------------------------------------------------------------------------------ kept rows in place
class Keep:
    def __init__(self, lens, H=2, ratio=0.4, block=0, seed=0, extra=5):
        import torch

        g = self.g = CH.rng(seed)
        B = len(lens)
        L = lib()
        self.lens, self.H, self.block = lens, H, block
        self.p = L.make_params(h_kv=H, group=1, n_ctx=max(lens), window=32, n_ctx_per_req=lens, n_sink=0, n_recent=0, budget_ratio=ratio)
        n_scores, n_kept, _ = L.kvsel_output_size(self.p)
        self.top = max(lens)
        self.scores = g.standard_normal(n_scores).astype(np.float32)
        idx, counts, offsets = [], [], []
        for n in lens:
            for _ in range(H):
                offsets.append(len(idx))
                k = int(np.floor(ratio * n))
                idx += sorted(g.choice(n, size=k, replace=False).tolist())
                counts.append(k)
        assert len(idx) == n_kept
        self.idx, self.counts, self.offsets = idx, counts, offsets
        rows = g.integers(0, 65536, (2, B, H, self.top, CH.D)).astype(np.uint16)
        self.rows = rows
        if block:
            nb = -(-self.top // block)
            self.table = g.permutation(B * nb).reshape(B, nb).astype(np.int32)
            pool = np.zeros((2, B * nb, block, H, CH.D), np.uint16)
            for b in range(B):
                x = np.zeros((2, nb * block, H, CH.D), np.uint16)
                x[:, :self.top] = rows[:, b].transpose(0, 2, 1, 3)
                pool[:, self.table[b]] = x.reshape(2, nb, block, H, CH.D)
            self.k, self.v = (torch.from_numpy(x.view(np.int16)).cuda() for x in pool)
            self.d_table = SH.ints(self.table)
            self.kv = L.make_kv_paged(self.k, self.v, self.d_table)
        else:
            wide = np.full((2, B, H, self.top, CH.D + 8), 9, np.uint16)
            wide[..., :CH.D] = rows
            self.k, self.v = (torch.from_numpy(x.view(np.int16)).cuda()[..., :CH.D] for x in wide)
            self.kv = L.make_kv_contiguous(self.k, self.v)
        self.cap = self.top + extra
        self.t = dict(idx=SH.ints(idx + [0]), counts=SH.ints(counts), offsets=torch.tensor(offsets, dtype=torch.int64, device="cuda"),
                      lens=SH.ints(np.full((B, H), 7)), seen=SH.ints(np.full((B, H), 7)), pos=SH.ints(np.full((B, H, self.cap), 7)),
                      acc=torch.full((B, H, self.cap), 7.0, device="cuda"), scores=torch.from_numpy(self.scores).cuda())
        self.ws = CH.workspace(1 << 17)

    def call(self, acc=True, scores=True):
        t = self.t
        lib().kvsel_compact_in_place(self.p, self.kv, t["idx"], t["counts"], t["offsets"], t["lens"], t["seen"], t["pos"], self.ws,
                                     scores=t["scores"] if scores else None, acc=t["acc"] if acc else None)
        return CH.status(self.ws)

    def cache(self):
        """[2][B][H][top][d] as the device has it."""
        x = [y.cpu().numpy().view(np.uint16) for y in (self.k.contiguous(), self.v.contiguous())]
        if not self.block:
            return np.stack(x)
        return np.stack([y[self.table].reshape(len(self.lens), -1, self.H, CH.D)[:, :self.top].transpose(0, 2, 1, 3) for y in x])

    def check(self, scores=True):
        got, pos, acc = self.cache(), self.t["pos"].cpu().numpy(), self.t["acc"].cpu().numpy()
        at = 0
        for b, n in enumerate(self.lens):
            for h in range(self.H):
                s = b * self.H + h
                kept = self.idx[self.offsets[s]:self.offsets[s] + self.counts[s]]
                where = SO.keep_rows(n, kept)
                want = self.rows[:, b, h].copy()
                want[:, :len(where)] = self.rows[:, b, h][:, where]
                assert np.array_equal(got[:, b, h], want), (b, h)
                assert pos[b, h, :len(where)].tolist() == where and (pos[b, h, len(where):] == 7).all()
                sc = self.scores[at:at + n][where] if scores else np.zeros(len(where), np.float32)
                assert np.array_equal(acc[b, h, :len(where)], sc) and (acc[b, h, len(where):] == 7).all()
                at += n
        assert np.array_equal(self.t["lens"].cpu().numpy().reshape(-1), self.counts)
        assert np.array_equal(self.t["seen"].cpu().numpy(), np.repeat(np.array(self.lens)[:, None], self.H, 1))


@pytest.mark.parametrize("block", [0, 8, 16, 32, 64])
@pytest.mark.parametrize("ratio", [0.0, 0.02, 0.4, 0.5, 0.93, 1.0])
def test_keep(block, ratio):
    c = Keep([1000, 33, 0, 64, 4099], ratio=ratio, block=block, seed=block)
    assert c.call() == 0
    c.check()


def test_keep_one_end():
    # all of the first rows, all of the last
    for last in (False, True):
        c = Keep([300, 64], ratio=0.5, block=16, seed=1)
        for s, n in enumerate([300, 300, 64, 64]):
            k = c.counts[s]
            c.idx[c.offsets[s]:c.offsets[s] + k] = list(range(n - k, n)) if last else list(range(k))
        c.t["idx"].copy_(SH.ints(c.idx + [0]))
        assert c.call() == 0
        c.check()


def test_keep_without_scores():
    c = Keep([500], H=3, seed=2)
    assert c.call(scores=False) == 0
    c.check(scores=False)
    c = Keep([500], H=3, seed=2)
    assert c.call(acc=False) == 0
    assert float(c.t["acc"].min()) == 7.0


def test_keep_records_what_is_wrong():
    for what in range(4):
        c = Keep([400, 200], ratio=0.3, block=16, seed=what)
        before = c.cache()
        if what == 0:
            c.t["idx"][5] = 400
        elif what == 1:
            c.t["idx"][c.counts[0] - 1] = -9
        elif what == 2:
            c.t["counts"][0] = 401
        else:
            c.t["offsets"][0] = 2 ** 62
        assert c.call() == -7
        got = c.cache()
        # the other segments are as they should be, and so is the first where nothing of it was moved
        for s in (1, 2, 3):
            b, h = divmod(s, 2)
            where = SO.keep_rows(c.lens[b], c.idx[c.offsets[s]:c.offsets[s] + c.counts[s]])
            assert np.array_equal(got[:, b, h, :len(where)], before[:, b, h][:, where])
        if what >= 2:
            assert np.array_equal(got[:, 0, 0], before[:, 0, 0]) and int(c.t["lens"][0, 0]) == 0
    c = Keep([400], ratio=0.3, block=16, seed=3)
    c.d_table[0, :] = -5
    before = c.cache()
    assert c.call() == -7
    assert np.array_equal(c.cache(), before)
