"""kvsel_attend against the fp64 oracle: single tokens and chunks, every cache layout, lengths
from nothing to many tiles, windows with first tokens, and the running weights."""
import numpy as np
import pytest

from tests import cache_harness as CH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    from kv_cache_eviction_window_gb300 import binding

    binding.load()
    yield


def run(acc=True, **kw):
    c = CH.Case(**kw).upload()
    ws = c.call(acc=acc)
    assert CH.status(ws) == 0
    c.check(acc=acc)
    return c


@pytest.mark.parametrize("layout,block", [("contiguous", 0), ("packed", 0), ("paged", 8), ("paged", 16), ("paged", 32),
                                          ("paged", 64)])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 300, 1111])
def test_single_tokens(layout, block, n):
    run(layout=layout, block=block, lens=n, H=2, G=4, seed=n)


@pytest.mark.parametrize("layout,block", [("contiguous", 0), ("paged", 8), ("paged", 32)])
@pytest.mark.parametrize("n", [0, 1, 63, 65, 300, 1111, 4000])
def test_single_tokens_with_room_for_more(layout, block, n):
    # rows in use far below max_len: the work is cut over the whole grid, whatever the length
    run(layout=layout, block=block, lens=n, H=2, G=4, pad_rows=4500, seed=n)


@pytest.mark.parametrize("pad_rows", [0, 9000])
def test_few_rows_of_every_kind(pad_rows):
    # the same calls where an item belongs to one cluster, and where the whole grid shares the work
    kw = dict(layout="paged", block=16, pad_rows=pad_rows)
    run(B=5, H=2, G=4, m=1, lens=[0, 1, 64, 513, 700], new=[0, 1, 1, 0, 1], seed=1, **kw)
    run(B=2, H=3, G=5, m=3, lens=[2, 517], per_head=False, seed=2, **kw)
    run(B=3, H=2, G=4, m=4, lens=[1, 300, 640], causal=False, seed=3, **kw)
    run(B=2, H=2, G=8, m=2, lens=[900, 65], window=70, n_sink=3, seed=4, **kw)
    run(B=7, H=8, G=2, m=8, lens=20 + 97 * np.arange(7), token_major=True, seed=5, **kw)
    run(B=38, H=8, G=1, m=1, lens=1 + 5 * np.arange(38), seed=6, **kw)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 13, 16, 17, 32, 100, 128])
def test_groups(G):
    run(G=G, H=1, lens=333, seed=G)


@pytest.mark.parametrize("m", [2, 3, 5, 16, 17, 31, 64, 65, 128, 200, 257])
@pytest.mark.parametrize("G,layout", [(1, "contiguous"), (4, "paged"), (7, "packed")])
def test_chunks(G, layout, m):
    run(G=G, H=2, m=m, lens=m + 190, layout=layout, seed=m)


@pytest.mark.parametrize("m,G", [(1, 3), (40, 7), (129, 1), (300, 4)])
def test_a_chunk_that_is_the_whole_cache(m, G):
    run(m=m, G=G, lens=m, layout="paged", block=8, seed=m)


@pytest.mark.parametrize("layout", ["contiguous", "paged", "packed"])
@pytest.mark.parametrize("m,G", [(1, 4), (6, 7), (50, 4), (130, 2)])
def test_ragged_batches(layout, m, G):
    g = CH.rng(m)
    new = g.integers(0, m + 1, 5)
    lens = np.array([0, 1, 700, 64, 259]) + new
    lens[0] = 0
    run(B=5, H=2, G=G, m=m, new=new, lens=lens if layout != "packed" else np.repeat(lens[:, None], 2, 1), layout=layout,
        token_major=True, seed=m)


def test_lengths_per_head():
    g = CH.rng(3)
    for m, layout in ((1, "contiguous"), (3, "paged"), (40, "paged"), (70, "contiguous")):
        run(B=3, H=4, G=4, m=m, lens=g.integers(m, 900, (3, 4)), per_head=True, layout=layout, pad_rows=5, seed=m)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 4), (5, 1), (16, 4), (100, 64), (128, 200), (1000, 4), (4096, 0),
                                           (50, 1000)])
@pytest.mark.parametrize("m,G,layout,block", [(1, 4, "paged", 16), (1, 8, "contiguous", 0), (9, 3, "paged", 64),
                                              (70, 4, "paged", 8), (300, 2, "contiguous", 0)])
def test_windows(window, n_sink, m, G, layout, block):
    run(B=2, H=2, G=G, m=m, lens=[1201, m + 7], window=window, n_sink=n_sink, layout=layout, block=block, seed=window)


@pytest.mark.parametrize("window,n_sink", [(3, 0), (57, 4), (256, 256), (700, 300)])
@pytest.mark.parametrize("m,G,layout,block", [(40, 1, "paged", 8), (70, 4, "contiguous", 0), (300, 2, "paged", 64)])
def test_windows_in_long_caches(window, n_sink, m, G, layout, block):
    # blocks of cached rows that no token sees lie between the first rows and the window, and before it
    run(B=3, H=2, G=G, m=m, new=[m, 1, m // 2], lens=[9001, 5 * 1024, 300], window=window, n_sink=n_sink, layout=layout,
        block=block, seed=window)


@pytest.mark.parametrize("m,G", [(1, 4), (5, 3), (90, 4)])
def test_every_row_visible(m, G):
    # the new tokens are not in the cache: every token sees all rows, an empty cache none
    run(B=3, G=G, m=m, lens=[0, 77, 500], causal=False, seed=m)


@pytest.mark.parametrize("m,G", [(4, 4), (40, 4), (150, 2)])
def test_fewer_rows_than_tokens(m, G):
    # tokens in front of the cache see nothing: zeros, and a log-sum-exp of -inf
    run(B=3, G=G, m=m, lens=[0, 1, m - 2], seed=m)


def test_scale_and_far_logits():
    run(lens=700, scale=1.0, logit=3.0, seed=1)                 # a softmax of almost one row
    run(lens=700, scale=1e-3, seed=2)                           # an almost even one
    run(lens=700, m=40, scale=0.5, logit=3.0, seed=3)
    # logits that rise along the cache: the running maximum moves in every tile
    for m in (1, 40):
        c = CH.Case(lens=1500, m=m, H=1, seed=4)
        c.k[0][0] = CH.bf16(c.k[0][0] + np.linspace(0, 4, 1500)[:, None] * c.q[0, 0, 0, 0][None])
        c.upload()
        ws = c.call(acc=True)
        assert CH.status(ws) == 0
        c.check(acc=True)


def test_work_cut_over_many_blocks():
    # one long segment, and many short ones: pieces of one item in many places, many items in one
    run(H=1, G=8, lens=20011, seed=1)
    run(B=64, H=8, G=4, lens=np.arange(64) * 5 + 1, layout="paged", seed=2, acc=False)
    run(B=300, H=2, G=2, lens=np.arange(300) % 7, seed=3)
    run(B=2, H=2, G=4, m=100, lens=[5000, 130], layout="paged", seed=4)
    # a few tiles each, of more segments than there are blocks: most blocks begin and end within one
    run(B=40, H=8, G=4, m=70, lens=70 + np.arange(40) * 9, layout="paged", seed=5)
    run(B=6, H=3, G=8, m=9, lens=[9, 40, 700, 1, 5000, 128], seed=6)
    # room for far more rows, and tokens, than there are: segments that end in many empty items
    run(B=40, H=4, G=4, m=40, lens=40 + np.arange(40) * 9, pad_rows=20000, layout="paged", block=64, seed=7)
    run(B=5, H=2, G=4, m=700, new=[0, 3, 700, 1, 90], lens=[0, 3, 900, 5000, 90], seed=8)
    # items of many pieces, few rows and many, and two pieces
    run(H=2, G=5, m=20, lens=12000, seed=9)
    run(H=3, G=4, m=130, lens=6000, seed=10)
    run(B=2, H=8, G=3, m=150, lens=[2500, 2300], layout="paged", block=32, seed=11)


@pytest.mark.parametrize("pad_rows", [0, 9000])
@pytest.mark.parametrize("m,G", [(6, 4), (32, 4), (70, 3), (300, 2)])
def test_few_rows_under_a_chunk(m, G, pad_rows):
    # the same calls where an item belongs to one block, and where the whole grid shares the work
    kw = dict(m=m, G=G, layout="paged", block=16, pad_rows=pad_rows, seed=m)
    run(B=4, H=2, new=[0, 1, m, m - 1], lens=[0, 1, m + 190, 513], **kw)
    run(B=2, H=2, lens=[m + 70, m], window=40, n_sink=3, **kw)
    run(B=2, H=3, lens=[130, m - 3], causal=False, per_head=False, **kw)


def test_weights_add_up_over_calls_and_results_repeat():
    import torch

    for m in (1, 33):
        c = CH.Case(lens=900, m=m, B=2, seed=m).upload()
        ws = c.call(acc=True)
        first = c.t["out"].clone(), c.t["acc"].clone()
        c.call(acc=True, ws=ws)
        assert torch.equal(first[0], c.t["out"])
        c.check(acc=True, calls=2)
        # without acc and lse: the same outputs
        c.call(acc=False, lse=False)
        assert torch.equal(first[0], c.t["out"])
        c.t["acc"].zero_()
        c.call(acc=True)
        assert torch.equal(first[1], c.t["acc"])


@pytest.mark.parametrize("m,G", [(1, 7), (6, 7), (100, 7), (200, 3)])
def test_a_result_does_not_depend_on_the_rest_of_the_batch(m, G):
    # (groups that do not fill a tile; logits that make the running maxima move)
    import torch

    c = CH.Case(B=2, G=G, H=1, m=m, lens=[900, 900], scale=0.6, seed=m).upload()
    c.call(acc=True)
    first = c.t["out"].clone(), c.t["lse"].clone(), c.t["acc"].clone()
    for _ in range(5):
        junk = torch.randn(1 << 22, device="cuda") * 1e30      # another content of the shared memories
        (junk.view(2048, 2048) @ junk.view(2048, 2048)).sum()
        c.t["acc"].zero_()
        c.t["q"][1] *= 1.25
        c.call(acc=True)
        for x, y in zip(first, (c.t["out"], c.t["lse"], c.t["acc"])):
            assert torch.equal(x[0], y[0])


@pytest.mark.parametrize("m,G,H,block", [(6, 7, 4, 32), (1, 7, 4, 32), (70, 7, 2, 16), (20, 1, 8, 64)])
def test_back_to_back_calls_repeat_bit_for_bit(m, G, H, block):
    # ragged lengths, calls without a pause: the warps of a CTA drift apart in every way
    import torch

    c = CH.Case(B=4, G=G, H=H, m=m, lens=[3001, 1900, 517, 2222], layout="paged", block=block, seed=m).upload()
    ws = c.call()
    first = c.t["out"].clone(), c.t["lse"].clone()
    for _ in range(20):
        for _ in range(50):
            c.call(ws=ws)
        assert CH.status(ws) == 0
        assert torch.equal(first[0], c.t["out"]) and torch.equal(first[1], c.t["lse"])
    c.check()


def test_lengths_are_read_by_a_captured_call():
    import torch

    c = CH.Case(lens=[900, 650], B=2, m=2, per_head=False, seed=5).upload()
    from kv_cache_eviction_window_gb300 import binding as L

    ws = CH.workspace(L.kvsel_attend_workspace_size(L.make_attn_params(**c.params), True))
    lens = c.t["lens"].clone()
    c.t["lens"].fill_(3)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.call(acc=True, ws=ws, stream=s)
        with torch.cuda.graph(g, stream=s):
            c.call(acc=True, ws=ws, stream=torch.cuda.current_stream())
    torch.cuda.current_stream().wait_stream(s)
    c.t["acc"].zero_()
    c.t["lens"].copy_(lens)
    g.replay()
    assert CH.status(ws) == 0
    c.check(acc=True)


def test_calls_side_by_side():
    import torch

    cases = [CH.Case(lens=3000 + 100 * i, H=2, m=1 + 40 * (i % 2), seed=i).upload() for i in range(4)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    from kv_cache_eviction_window_gb300 import binding as L

    wss = [CH.workspace(L.kvsel_attend_workspace_size(L.make_attn_params(**c.params), True)) for c in cases]
    torch.cuda.synchronize()
    for c, s, ws in zip(cases, streams, wss):
        c.call(acc=True, ws=ws, stream=s)
    torch.cuda.synchronize()
    for c, ws in zip(cases, wss):
        assert CH.status(ws) == 0
        c.check(acc=True)


def test_bad_lengths_blocks_and_offsets_are_reported():
    import torch

    for m in (1, 40):
        c = CH.Case(lens=200, m=m, layout="paged", seed=1).upload()
        ora = c.oracle()
        c.t["lens"].fill_(c.max_len + 9)        # clamped to max_len
        ws = c.call(acc=True)
        assert CH.status(ws) == -7
        c.check(ora, acc=True)
        c.t["lens"].fill_(-4)                    # counts as empty
        ws = c.call(ws=ws)
        assert CH.status(ws) == -7
        assert torch.all(c.t["out"] == 0) and torch.all(torch.isneginf(c.t["lse"]))
        # a block out of range: its rows read as zeros
        c = CH.Case(lens=200, m=m, layout="paged", seed=1)
        for h in range(c.H):
            c.k[0][h][48:64] = 0.0
            c.v[0][h][48:64] = 0.0
        c.upload()
        c.keep[2][0, 3] = c.keep[2].numel() + 5
        ws = c.call(acc=True)
        assert CH.status(ws) == -7
        c.check(acc=True)
        c = CH.Case(lens=200, m=m, layout="packed", seed=2).upload()
        c.offsets[1] += 1                         # the last segment would end one row too late
        ws = c.call()
        assert CH.status(ws) == -7
        out = CH.to_f64(c.t["out"]).reshape(1, c.H, c.G, m, CH.D)
        assert np.all(out[0, 1] == 0)
        assert np.isfinite(out).all()


def test_attention_over_what_a_layer_call_kept():
    """run_layer's compacted cache goes straight into the attention: the query tokens attend to
    the kept rows only, and to the whole cache when everything is kept."""
    import torch

    from kv_cache_eviction_window_gb300 import binding as L
    from kv_cache_eviction_window_gb300 import datagen
    from oracle import cache_oracle as CO
    from tests import gpu_harness as GH

    wl = datagen.WORKLOADS[3].replace(layers=1, h_kv=2, window=32)
    inp = datagen.make_layer(wl, 0, n_ctx=2500)
    p = L.params_from_workload(wl, n_ctx=2500)
    q, k, v = (GH.torch_bf16(x) for x in (inp["q"], inp["k"][0], inp["v"][0]))
    buf = L.LayerBuffers(p)
    L.kvsel_run_layer(p, q, L.make_kv_contiguous(k, v), None, buf.s_attn, buf.s_val, buf.idx, buf.counts, buf.offsets,
                      buf.k_out, buf.v_out, buf.ws)
    G, W = wl.group, 3
    pa = L.make_attn_params(h_kv=2, group=G, batch=1, n_new=W, max_len=2500, causal=False, n_rows=buf.n_kept)
    out = torch.empty((1, 2 * G, W, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((1, 2 * G, W), device="cuda")
    # (scoring and attention calls take turns on one workspace)
    ws = CH.workspace(max(L.kvsel_attend_workspace_size(pa), L.kvsel_workspace_size(p)))
    qn = q.reshape(1, 2 * G, 32, 128)[:, :, -W:].contiguous()
    for _ in range(2):
        L.kvsel_attend(pa, qn, L.make_kv_packed(buf.k_out, buf.v_out), buf.counts, out, ws, offsets=buf.offsets, lse=lse)
        L.kvsel_run_layer(p, q, L.make_kv_contiguous(k, v), None, buf.s_attn, buf.s_val, buf.idx, buf.counts, buf.offsets,
                          buf.k_out, buf.v_out, ws)
    assert CH.status(ws) == 0
    counts, offs = buf.counts.cpu().numpy(), buf.offsets.cpu().numpy()
    for h in range(2):
        idx = buf.idx.cpu().numpy()[offs[h]:offs[h] + counts[h]]
        o = CO.attend_segment(CH.to_f64(qn)[0, h * G:(h + 1) * G], CH.to_f64(k)[h][idx], CH.to_f64(v)[h][idx], causal=False)
        e = 132 * 2.0 ** -23 * o["abs_logit"] + 2.0 ** -14
        tol = (2 * e[..., None] + 2.0 ** -8) * o["mean_abs"] + 2.0 ** -8 * np.abs(o["out"])
        assert np.all(np.abs(CH.to_f64(out)[0, h * G:(h + 1) * G] - o["out"]) <= tol)


@pytest.mark.parametrize("G,m", [(100, 3), (128, 5), (65, 9), (43, 8), (3, 400)])
def test_wide_groups_in_chunks(G, m):
    # groups that fill a tile alone, or leave most of one empty
    run(G=G, m=m, H=2, lens=[m + 301], layout="paged", block=16, seed=G)


@pytest.mark.parametrize("m,G,acc", [(6, 7, False), (300, 4, False), (300, 4, True)])
def test_a_wait_that_runs_out_is_reported(m, G, acc):
    """wait_cycles = 1 makes every wait that is not already satisfied give up: the call ends with
    KVSEL_ETIMEOUT in the status word, and the next call on the same workspace is sound."""
    import torch

    c = CH.Case(B=2, G=G, H=2, m=m, lens=[2000, 900], layout="paged", seed=m).upload()
    good = dict(c.params)
    c.params["wait_cycles"] = 1
    ws = c.call(acc=acc)
    assert CH.status(ws) == -6
    c.params = good
    c.t["out"].fill_(7.0)
    c.t["lse"].fill_(7.0)
    c.t["acc"].zero_()
    c.call(acc=acc, ws=ws)
    assert CH.status(ws) == 0
    c.check(acc=acc)
    torch.cuda.synchronize()


def test_a_workspace_elsewhere_is_refused():
    from kv_cache_eviction_window_gb300 import binding as L

    c = CH.Case(lens=50).upload()
    ws = CH.workspace(L.kvsel_attend_workspace_size(L.make_attn_params(**c.params), True))
    with pytest.raises(L.KvselError) as e:
        c.call(acc=True, ws=ws.cpu())
    assert e.value.code == L.KVSEL_EINVAL
    c.call(acc=True, ws=ws)
    c.check(acc=True)


def test_more_blocks_than_can_be_planned_are_refused():
    from kv_cache_eviction_window_gb300 import binding as L

    p = dict(h_kv=64, group=4, batch=512, n_new=40, acc_stride=1 << 30)
    with pytest.raises(L.KvselError) as e:
        L.kvsel_attend_workspace_size(L.make_attn_params(max_len=1 << 30, **p), True)
    assert e.value.code == L.KVSEL_EUNSUPPORTED
    # without weights, or with a window, there are few
    assert L.kvsel_attend_workspace_size(L.make_attn_params(max_len=1 << 30, **p), False) > 0
    assert L.kvsel_attend_workspace_size(L.make_attn_params(max_len=1 << 30, window=4096, **p), True) > 0


@pytest.mark.parametrize("m", [1, 40])
def test_caches_beyond_2_to_the_32_elements(m):
    """Blocks and rows whose element offset passes 32 bits, in a paged and in a packed cache, and a
    token-major contiguous one ([token][head][d])."""
    import torch

    from kv_cache_eviction_window_gb300 import binding as L

    G, H, n, bs = 4, 4, 200, 16
    c = CH.Case(G=G, H=H, m=m, lens=n, seed=m)
    ora = c.oracle()
    q = CH.to_gpu_bf16(c.q.reshape(1, H * G, m, CH.D))
    k, v = (CH.to_gpu_bf16(np.stack(x[0])) for x in (c.k, c.v))          # [H][n][d]
    blocks = (1 << 32) // (bs * H * CH.D) + 64
    pools = [torch.empty((blocks, bs, H, CH.D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    used = -(-n // bs)
    table = torch.arange(blocks - used, blocks, dtype=torch.int32, device="cuda").flip(0).reshape(1, used).contiguous()
    for pool, x in zip(pools, (k, v)):
        rows = torch.zeros((used * bs, H, CH.D), dtype=torch.bfloat16, device="cuda")
        rows[:n] = x.permute(1, 0, 2)
        pool[table[0].long()] = rows.view(used, bs, H, CH.D)
    flat = [p.view(-1, CH.D) for p in pools]                             # the same memory as packed rows
    base = flat[0].shape[0] - H * n
    packed = [x.clone() for x in (k, v)]
    strided = [torch.empty((n, H, CH.D), dtype=torch.bfloat16, device="cuda").copy_(x.permute(1, 0, 2)) for x in (k, v)]
    for kind in ("paged", "strided", "packed"):
        p = L.make_attn_params(h_kv=H, group=G, batch=1, n_new=m, max_len=n, n_rows=flat[0].shape[0] if kind == "packed" else 0,
                               acc_stride=n, lens_per_head=kind == "packed")
        offsets = None
        if kind == "paged":
            kv = L.make_kv_paged(pools[0], pools[1], table)
        elif kind == "strided":
            kv = L.make_kv_contiguous(*(x.permute(1, 0, 2) for x in strided))
        else:
            for f, x in zip(flat, packed):
                f[base:] = x.reshape(H * n, CH.D)
            offsets = torch.arange(H, device="cuda", dtype=torch.int64) * n + base
            kv = L.make_kv_packed(flat[0], flat[1])
        lens = torch.full((H,) if kind == "packed" else (1,), n, dtype=torch.int32, device="cuda")
        c.t = dict(out=torch.empty((1, H * G, m, CH.D), dtype=torch.bfloat16, device="cuda"),
                   lse=torch.empty((1, H * G, m), device="cuda"), acc=torch.zeros((1, H, n), device="cuda"))
        ws = CH.workspace(L.kvsel_attend_workspace_size(p, True))
        L.kvsel_attend(p, q, kv, lens, c.t["out"], ws, offsets=offsets, lse=c.t["lse"], acc=c.t["acc"])
        assert CH.status(ws) == 0
        c.check(ora, acc=True)
