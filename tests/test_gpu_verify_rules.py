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
