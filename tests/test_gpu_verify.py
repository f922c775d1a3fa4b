"""kvsel_verify against exact rational arithmetic: every mode and type, chains, stars and trees, ragged
requests, and what is refused or recorded."""
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


def run(pad=0, lead=0, **kw):
    c = SH.VerifyCase(**kw).upload(pad=pad, lead=lead)
    assert CH.status(c.call()) == 0
    c.check()
    return c


@pytest.mark.parametrize("mode", ["sampled", "point", "greedy"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["chain", "star", "tree"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 5003])
def test_modes(mode, dtype, kind, V):
    for seed in range(3):
        run(B=4, m=9, V=V, mode=mode, dtype=dtype, kind=kind, seed=seed)


@pytest.mark.parametrize("mode", ["sampled", "point", "greedy"])
@pytest.mark.parametrize("m", [1, 2, 31, 33, 64, 300])
def test_nodes(mode, m):
    run(B=3, m=m, V=211, mode=mode, seed=m, new=[m, max(1, m // 2), 0], near=0.2)


@pytest.mark.parametrize("near", [0.0, 0.05, 3.0])
@pytest.mark.parametrize("zeros", [0.0, 0.5])
def test_close_and_far_drafts(near, zeros):
    # the same distribution: nothing is left of the rest after a rejection; far ones: long runs of rejections
    for kind in ("star", "tree"):
        run(B=8, m=24, V=64, near=near, zeros=zeros, kind=kind, seed=int(near * 10), sharp=1.0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V,pad,lead", [(1001, 3, 0), (1001, 0, 1), (64, 7, 5), (1000, 24, 8)])
def test_strides_and_alignment(dtype, V, pad, lead):
    run(B=2, m=5, V=V, dtype=dtype, pad=pad, lead=lead, seed=V)
    run(B=2, m=5, V=V, dtype=dtype, mode="greedy", pad=pad, lead=lead, seed=V)


def test_draft_on_another_boundary_than_target():
    c = SH.VerifyCase(B=2, m=6, V=1003, kind="star", near=2.0, seed=4).upload()
    d = SH.VerifyCase(B=2, m=6, V=1003, kind="star", near=2.0, seed=4).upload(lead=1)
    c.t["draft"] = d.t["draft"]
    assert CH.status(c.call()) == 0
    c.check()


@pytest.mark.parametrize("mode,dtype,near,pad,lead", [("sampled", "fp32", 0.1, 0, 0), ("sampled", "bf16", 2.0, 5, 3), ("point", "bf16", 0.1, 1, 1),
                                                      ("point", "fp32", 0.1, 2, 1)])
def test_draws_all_over_long_rows(mode, dtype, near, pad, lead):
    # many requests: a CTA has a row to itself, a warp several stretches of it; the draws fall all over them
    run(B=230, m=3, V=9001, mode=mode, dtype=dtype, kind="star", near=near, pad=pad, lead=lead, sharp=0.5, seed=pad)


def test_draws_where_rows_do_not_share_a_boundary():
    c = SH.VerifyCase(B=230, m=2, V=9001, kind="star", near=2.0, seed=6, sharp=0.5).upload()
    d = SH.VerifyCase(B=230, m=2, V=9001, kind="star", near=2.0, seed=6, sharp=0.5).upload(lead=1)
    c.t["draft"] = d.t["draft"]
    assert CH.status(c.call()) == 0
    c.check()


def test_large_vocabulary():
    c = SH.VerifyCase(B=1, m=4, V=262144, kind="star", near=1.0, seed=2).upload()
    assert CH.status(c.call()) == 0
    c.check()


@pytest.mark.parametrize("u0", [0.0, 1.0 - 2.0 ** -24, 0.5, 2.0 ** -30])
def test_the_draw_at_its_ends(u0):
    for mode, zeros in (("sampled", 0.6), ("point", 0.6)):
        c = SH.VerifyCase(B=6, m=4, V=500, mode=mode, kind="star", near=2.0, zeros=zeros, seed=9)
        c.u[:, 0] = u0
        c.upload()
        assert CH.status(c.call()) == 0
        c.check()


def test_tests_at_their_ends():
    # u = 0 accepts what has any probability, u just below 1 what the target likes at least as much
    for u in (0.0, 1.0 - 2.0 ** -24):
        c = SH.VerifyCase(B=6, m=7, V=40, kind="star", seed=3, zeros=0.3)
        c.u[:, 1:] = u
        c.upload().call()
        c.check()


def test_the_same_token_twice():
    # siblings with one token: after its rejection a point draft has no weight left
    c = SH.VerifyCase(B=3, m=6, V=50, mode="point", kind="star", seed=1)
    c.tokens[:, 1:] = c.tokens[:, 1:2]
    c.u[:, 1:] = 0.999
    c.upload().call()
    c.check()


def test_no_mass():
    c = SH.VerifyCase(B=2, m=3, V=30, mode="point", kind="star", seed=1)
    c.p[0] = 0.0
    c.upload()
    assert CH.status(c.call()) == 0
    c.check()
    assert c.t["next"].tolist()[0] == -1


def test_not_a_number_counts_as_nothing():
    c = SH.VerifyCase(B=2, m=4, V=300, kind="star", near=1.0, seed=6)
    c.p[:, 0, 5:9] = 0.0
    c.q[:, 0, 20:22] = 0.0
    want = c.oracle()
    c.p[:, 0, 5:9] = np.nan
    c.q[:, 0, 20:22] = np.nan
    c.upload().call()
    c.check(want)
    c = SH.VerifyCase(B=2, m=4, V=300, mode="greedy", kind="star", near=0.1, seed=6)
    c.p[:, 0, 5:90] = np.nan
    c.p[1, 0, 100:110] = np.inf
    c.upload().call()
    c.check()


def test_ties_go_to_the_lowest_token():
    c = SH.VerifyCase(B=4, m=5, V=6000, mode="greedy", dtype="bf16", kind="star", seed=2)
    c.p[:] = -1.0
    c.p[0, :, 5999] = 2.0
    c.p[1, :, [10, 4000, 5999]] = 2.0
    c.p[2, :, [0, 1]] = 0.0
    c.p[2, :, 1] = -0.0
    c.tokens[1, 3], c.tokens[2, 2] = 10, 1
    c.upload().call()
    c.check()
    assert c.t["counts"].tolist()[1] == 2 and c.t["next"].tolist()[0] == 5999 and c.t["next"].tolist()[3] == 0


def test_what_is_recorded():
    for mode in ("sampled", "point", "greedy"):
        c = SH.VerifyCase(B=2, m=6, V=40, mode=mode, kind="star", seed=1)
        c.tokens[0, 2], c.tokens[1, 3] = 40, -1
        c.upload()
        assert CH.status(c.call()) == -7
        c.check()
    c = SH.VerifyCase(B=2, m=6, V=40, kind="chain", seed=1)
    c.parents[0, 3] = 3
    c.upload()
    assert CH.status(c.call()) == -7
    c.check()
    c = SH.VerifyCase(B=2, m=6, V=40, kind="chain", seed=1, new=[6, 6]).upload()
    c.t["new_lens"].copy_(SH.ints([9, 6]))
    assert CH.status(c.call()) == -7
    c.check()


def test_the_target_is_followed():
    # 40,000 requests of one drafted token: the first token's frequencies are the target's.  A frequency of n
    # draws is off by sqrt(p (1 - p) / n); 5 of those in 40 tokens happen in 2 of 10^5 runs.
    import torch

    V, total, seen = 10, 0, np.zeros(10)
    g = CH.rng(0)
    p, q = SH.probabilities(g, V).astype(np.float64), SH.probabilities(g, V).astype(np.float64)
    for turn in range(40):
        c = SH.VerifyCase(B=1000, m=3, V=V, kind="star", seed=turn)
        c.p[:, 0], c.q[:, 0] = p, q
        for b in range(1000):
            c.tokens[b, 1:] = np.searchsorted(np.cumsum(q), c.g.random(2) * q.sum(), side="right").clip(0, V - 1)
        c.upload().call()
        torch.cuda.synchronize()
        path, counts, nxt = (c.t[x].cpu().numpy() for x in ("path", "counts", "next"))
        first = np.where(counts > 1, c.tokens[np.arange(1000), np.maximum(path[:, 1], 0)], nxt)
        seen += np.bincount(first, minlength=V)
        total += 1000
    assert np.all(np.abs(seen / total - p) <= 5 * np.sqrt(p * (1 - p) / total) + 1e-9)


def test_streams_and_graphs():
    import torch

    cases = [SH.VerifyCase(B=40, m=12, V=3000, mode=mode, seed=3).upload() for mode in ("sampled", "point", "greedy")]
    streams = [torch.cuda.Stream() for _ in cases]
    wss = [CH.workspace(1 << 17) for _ in cases]
    torch.cuda.synchronize()
    for c, s, ws in zip(cases, streams, wss):
        c.call(ws=ws, stream=s)
    for c, ws in zip(cases, wss):
        assert CH.status(ws) == 0
        c.check()
    c = cases[0]
    g, s = torch.cuda.CUDAGraph(), streams[0]
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            c.call(ws=wss[0], stream=torch.cuda.current_stream())
    c.u = c.g.random(c.u.shape).astype(np.float32)
    c.t["u"].copy_(torch.from_numpy(c.u))
    g.replay()
    torch.cuda.synchronize()
    c.check()
