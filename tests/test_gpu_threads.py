"""Calls from host threads that have made no CUDA call before, several at once, each with a stream and a
workspace of its own."""
import threading

import numpy as np
import pytest

from kv_cache_eviction_window_gb300 import datagen
from tests import cache_harness as CH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    from kv_cache_eviction_window_gb300 import binding

    binding.load()
    yield


def in_threads(calls):
    """Runs the calls at once, each in a new thread; raises what one of them raised."""
    errors = []

    def run(call):
        try:
            call()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("m,G,acc", [(1, 4, True), (6, 4, False), (6, 7, True), (40, 4, True), (300, 2, False)])
@pytest.mark.parametrize("layout", ["contiguous", "paged", "packed"])
def test_attention_from_new_threads(layout, m, G, acc):
    import torch

    from kv_cache_eviction_window_gb300 import binding as L

    cases = [CH.Case(H=2, G=G, m=m, lens=1500 - 100 * i, layout=layout, seed=i).upload() for i in range(6)]
    oras = [c.oracle() for c in cases]
    wss = [CH.workspace(L.kvsel_attend_workspace_size(L.make_attn_params(**c.params), acc)) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()

    def work(c, ws, s):
        def call():
            for _ in range(20):
                c.call(ws=ws, stream=s)
            if acc:
                c.call(acc=True, ws=ws, stream=s)
        return call

    in_threads([work(c, ws, s) for c, ws, s in zip(cases, wss, streams)])
    torch.cuda.synchronize()
    for c, o, ws in zip(cases, oras, wss):
        assert CH.status(ws) == 0
        c.check(o, acc=acc)


@pytest.mark.parametrize("value_aware", [False, True])
def test_layer_calls_from_new_threads(value_aware):
    import torch

    from kv_cache_eviction_window_gb300 import binding as L
    from tests import gpu_harness as GH

    wl = datagen.WORKLOADS[2].replace(layers=1, h_kv=2)
    n = 900
    inp = datagen.make_layer(wl, 0, n_ctx=n)
    p = L.params_from_workload(wl, n_ctx=n, value_aware=int(value_aware), concurrent=1)
    q, k, v = (GH.torch_bf16(x) for x in (inp["q"], inp["k"][0], inp["v"][0]))
    w = GH.torch_bf16(inp["w_o"]) if value_aware else None
    kv = L.make_kv_contiguous(k, v)
    bufs, streams = [L.LayerBuffers(p) for _ in range(5)], [torch.cuda.Stream() for _ in range(5)]

    def layer(b, s):
        L.kvsel_run_layer(p, q, kv, w, b.s_attn, b.s_val, b.idx, b.counts, b.offsets, b.k_out, b.v_out, b.ws, stream=s)

    layer(bufs[0], None)
    torch.cuda.synchronize()
    in_threads([lambda b=b, s=s: layer(b, s) for b, s in zip(bufs[1:], streams[1:])])
    torch.cuda.synchronize()
    for b in bufs:
        assert L.kvsel_get_device_status(b.ws) == 0
        assert torch.equal(b.idx, bufs[0].idx) and torch.equal(b.k_out, bufs[0].k_out)
    assert np.all(bufs[0].counts.cpu().numpy() > 0)
