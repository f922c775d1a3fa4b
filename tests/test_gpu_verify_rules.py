"""kvsel_verify's promises away from the ordinary call: waits that run out, probabilities that sum to more than one, tensors
of other shapes."""
import functools

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


def with_wait(c, cycles, monkeypatch, **kw):
    from kv_cache_eviction_window_gb300 import binding as L

    with monkeypatch.context() as m:
        m.setattr(L, "make_verify_params", functools.partial(L.make_verify_params, wait_cycles=cycles))
        return c.call(**kw)


@pytest.mark.parametrize("mode", ["sampled", "point", "greedy"])
@pytest.mark.parametrize("B,V", [(1, 5000), (3, 40000), (12, 40000)])
def test_a_wait_that_runs_out(mode, B, V, monkeypatch):
    # clusters of 4 and of 16 CTAs, none of which has another's numbers when it first looks; the workspace serves on
    c = SH.VerifyCase(B=B, m=9, V=V, mode=mode, kind="star", near=2.0, seed=B).upload()
    ws = with_wait(c, 1, monkeypatch)
    assert CH.status(ws) == -6
    for _ in range(20):
        with_wait(c, 1, monkeypatch, ws=ws)
    assert CH.status(ws) == -6
    with_wait(c, 0, monkeypatch, ws=ws)
    assert CH.status(ws) == 0
    c.check()


def test_a_request_of_one_cta_waits_for_nobody(monkeypatch):
    c = SH.VerifyCase(B=2, m=6, V=1000, seed=1).upload()
    ws = with_wait(c, 1, monkeypatch)
    assert CH.status(ws) == 0
    c.check()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [8, 6000])
@pytest.mark.parametrize("u0,token", [(0.25, 0), (0.99, 0)])
def test_a_thousand_rejections_of_a_row_that_sums_to_more_than_one(dtype, V, u0, token):
    # 1023 siblings, each with a token that the target never takes, and a target row that sums to 17/16: the masses
    # before them sum to more than 1024.  Token 2 has 1/16 - 1024 * 2^-14 = 0 left by then, token 0 more than 1 - 1087 * 2^-16.
    from oracle import step_oracle as SO

    m = 1024
    c = SH.VerifyCase(B=1, m=2, V=8, kind="star", dtype=dtype, seed=1)
    c.m, c.V, c.new = m, V, np.array([m])
    c.p, c.q = np.zeros((1, m, V)), np.zeros((1, m, V))
    c.p[0, 0, [0, 2]] = 1.0, 2.0 ** -4
    c.q[0, 0, [0, 1, 2]] = 2.0 ** -16, 1.0, 2.0 ** -14
    c.parents, c.tokens = np.array([[-1] + [0] * (m - 1)]), np.ones((1, m), int)
    c.u = np.full((1, m), 0.5, np.float32)
    c.u[0, 0] = u0
    want = SO.verify(c.tokens[0].tolist(), c.parents[0].tolist(), c.p[0, :, :8], c.q[0, :, :8], c.u[0], "sampled")
    assert want == ([0], token)
    c.upload()
    assert CH.status(c.call()) == 0
    c.check([want])
