"""kvsel_rope and kvsel_rope_cache against the 64-bit oracle: layouts, part of the head, scalings, directions,
far positions, strides, in place, and the gradient."""
import numpy as np
import pytest

from oracle import step_oracle as SO
from tests import cache_harness as CH
from tests import step_harness as SH

pytestmark = pytest.mark.gpu
THETA = 500000.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    yield


def lib():
    from kv_cache_eviction_window_gb300 import binding

    return binding


def table(**kw):
    kw = dict(dict(theta=THETA, orig_len=8192), **kw)
    t = lib().kvsel_rope_table(**kw)
    f, scale = SO.frequencies(kw.get("rot_dim", 128), kw["theta"], kw.get("scaling", "none"), kw.get("factor", 1.0), kw["orig_len"])
    return t, dict(f=f, scale=kw.get("value_scale") or scale, interleaved=kw.get("layout") == "interleaved",
                   direction=kw.get("direction", "forward"))


def close(got, x, pos, o):
    """A turned value is x1 c - x2 s.  The angle, at most pi, is cut to 23 bits of a turn (2 pi 2^-23 < 7.5e-7) and made of
    them by one product and sum of rounded constants (4.5e-7 at most, over all of them); the approximate sine and cosine are
    off by 2^-21.19 < 4.2e-7 within [-pi, pi]; factor, product and sum round three times, 2^-24 each, 1.8e-7.  Together
    1.8e-6, below 2^-19 = 1.9e-6 of |x1| + |x2| times the factor.  (At positions near 2^31 the angles here, pos f rounded to
    64 bits, are off by 2^-22 themselves, what is left of the bound and as much again, if all of these met.)  One rounding
    to bf16: 2^-8 of the value."""
    want = SO.rope(x, pos, **o)
    rot = 2 * len(o["f"])
    half = rot // 2
    size = np.abs(x).copy()
    a, b = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if o["interleaved"] else (np.arange(half), np.arange(half, rot))
    grow = 1 / o["scale"] if o["direction"] == "inverse" else o["scale"]
    size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * grow
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * (1 + 2.0 ** -8) * size
    err = np.abs(got - want)
    assert np.all(err[..., :rot] <= tol[..., :rot]), float((err / np.maximum(tol, 1e-30))[..., :rot].max())
    assert np.array_equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [16, 32, 48, 64, 96, 112, 128])
@pytest.mark.parametrize("direction", ["forward", "transpose", "inverse"])
def test_parts_of_the_head(layout, rot, direction):
    t, o = table(layout=layout, rot_dim=rot, direction=direction, scaling="yarn", factor=4.0)
    g = CH.rng(rot)
    x, k, pos = CH.bf16(g.standard_normal((2, 5, 7, 128))), CH.bf16(g.standard_normal((2, 2, 7, 128))), g.integers(0, 5000, (2, 7))
    for inplace in (False, True):
        q, kk = CH.to_gpu_bf16(x), CH.to_gpu_bf16(k)
        qo, ko = (q, kk) if inplace else (CH.to_gpu_bf16(x * 0 + 3), CH.to_gpu_bf16(k * 0 + 3))
        lib().kvsel_rope(t, q, SH.ints(pos), q_out=None if inplace else qo, k=kk, k_out=None if inplace else ko)
        close(CH.to_f64(qo), x, pos[:, None], o)
        close(CH.to_f64(ko), k, pos[:, None], o)


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 8.0), ("ntk", 8.0), ("yarn", 16.0), ("yarn", 1.0), ("bands", 8.0)])
@pytest.mark.parametrize("far", [0, 1, 100, 2 ** 17, 2 ** 24 + 1, 2 ** 31 - 64])
def test_scalings_and_far_positions(scaling, factor, far):
    t, o = table(scaling=scaling, factor=factor)
    g = CH.rng(far % 1000)
    x, pos = CH.bf16(g.standard_normal((1, 3, 33, 128))), far + np.arange(33)[None]
    q = CH.to_gpu_bf16(x)
    lib().kvsel_rope(t, q, SH.ints(pos))
    close(CH.to_f64(q), x, pos[:, None], o)
    neg = -pos                                    # positions relative to later ones
    q = CH.to_gpu_bf16(x)
    lib().kvsel_rope(t, q, SH.ints(neg))
    close(CH.to_f64(q), x, neg[:, None], o)


@pytest.mark.parametrize("B,n,hq,hk", [(1, 1, 1, 0), (1, 1, 32, 8), (64, 1, 28, 4), (3, 517, 7, 1), (2, 1000, 40, 8), (1, 31, 9, 0)])
def test_shapes_and_slices(B, n, hq, hk):
    # slices of a projection's output, token-major; outputs head-major
    t, o = table()
    g = CH.rng(n)
    wide = CH.bf16(g.standard_normal((B, n, hq + 2 * hk, 128)))
    pos = g.integers(0, 10 ** 6, (B, n))
    w = CH.to_gpu_bf16(wide).transpose(1, 2)
    qo, ko = CH.to_gpu_bf16(np.zeros((B, hq, n, 128))), CH.to_gpu_bf16(np.zeros((B, max(hk, 1), n, 128)))
    x = wide.transpose(0, 2, 1, 3)
    if hk:
        lib().kvsel_rope(t, w[:, :hq], SH.ints(pos), q_out=qo, k=w[:, hq:hq + hk], k_out=ko)
        close(CH.to_f64(ko), x[:, hq:hq + hk], pos[:, None], o)
    else:
        lib().kvsel_rope(t, w[:, :hq], SH.ints(pos), q_out=qo)
    close(CH.to_f64(qo), x[:, :hq], pos[:, None], o)
    assert np.array_equal(CH.to_f64(w), x)
    # in place, positions in common, the values' heads untouched
    lib().kvsel_rope(t, w[:, :hq + hk], SH.ints(pos[0]))
    close(CH.to_f64(w)[:, :hq + hk], x[:, :hq + hk], pos[0][None, None], o)
    assert np.array_equal(CH.to_f64(w)[:, hq + hk:], x[:, hq + hk:])


def test_ragged_requests():
    t, o = table(layout="interleaved", rot_dim=64)
    g = CH.rng(1)
    x, pos, new = CH.bf16(g.standard_normal((4, 3, 9, 128))), g.integers(0, 100, (4, 9)), [9, 0, 4, 1]
    q, out = CH.to_gpu_bf16(x), CH.to_gpu_bf16(np.full((4, 3, 9, 128), 7.0))
    lib().kvsel_rope(t, q, SH.ints(pos), q_out=out, new_lens=SH.ints(new))
    got = CH.to_f64(out)
    for b, m in enumerate(new):
        close(got[b, :, :m], x[b, :, :m], pos[b, :m][None], o)
        assert (got[b, :, m:] == 7.0).all()


def test_there_and_back_and_the_gradient():
    # INVERSE undoes FORWARD; <R x, y> = <x, R^T y> with TRANSPOSE: the gradient of a sum weighted by y
    g = CH.rng(2)
    x, y, pos = CH.bf16(g.standard_normal((1, 2, 50, 128))), CH.bf16(g.standard_normal((1, 2, 50, 128))), g.integers(0, 10 ** 6, (1, 50))
    tables = {d: table(scaling="yarn", factor=8.0, direction=d)[0] for d in ("forward", "transpose", "inverse")}
    q, b, back = CH.to_gpu_bf16(x), CH.to_gpu_bf16(y), CH.to_gpu_bf16(x)
    lib().kvsel_rope(tables["forward"], q, SH.ints(pos))
    lib().kvsel_rope(tables["transpose"], b, SH.ints(pos))
    lib().kvsel_rope(tables["forward"], back, SH.ints(pos))
    lib().kvsel_rope(tables["inverse"], back, SH.ints(pos))
    # two roundings of 2^-8 of values no larger than the pair
    assert np.all(np.abs(CH.to_f64(back) - x) <= 2.1 * 2.0 ** -8 * (np.abs(x) + np.abs(np.roll(x, 64, -1))))
    one, two = (CH.to_f64(q) * y).sum(-1), (x * CH.to_f64(b)).sum(-1)
    assert np.all(np.abs(one - two) <= 2.0 ** -8 * 1.01 * ((np.abs(CH.to_f64(q)) * np.abs(y)).sum(-1) + (np.abs(x) * np.abs(CH.to_f64(b))).sum(-1)))
    # against differences: the map is linear, so a step in one column moves the result by the column of R
    f, scale = SO.frequencies(128, THETA, "yarn", 8.0, 8192)
    step = np.zeros((1, 2, 50, 128))
    step[..., 5] = 1.0
    col = SO.rope(step, pos[:, None], f, scale)
    grad = CH.to_f64(b)[..., 5]
    assert np.all(np.abs((col * y).sum(-1) - grad) <= 2.0 ** -8 * np.abs(grad) + 2.0 ** -19 * 4 * scale)


@pytest.mark.parametrize("block", [0, 8, 16, 64])
@pytest.mark.parametrize("per_head", [False, True])
def test_cached_keys(block, per_head):
    import torch

    t, o = table(direction="inverse", scaling="bands", factor=8.0)
    g = CH.rng(block)
    B, H, n = 3, 2, 301
    lens = np.array([[301, 17], [0, 200], [64, 65]]) if per_head else np.array([301, 0, 64])
    x, pos = CH.bf16(g.standard_normal((B, H, n, 128))), g.integers(-5, 10 ** 6, (B, H, n))
    if block:
        nb = -(-n // block)
        order = g.permutation(B * nb).reshape(B, nb)
        pool = np.full((B * nb, block, H, 128), 5.0)
        for b in range(B):
            rows = np.full((nb * block, H, 128), 5.0)
            rows[:n] = x[b].transpose(1, 0, 2)
            pool[order[b]] = rows.reshape(nb, block, H, 128)
        k, d_table = CH.to_gpu_bf16(pool), SH.ints(order)
        kv = lib().make_kv_paged(k, k, d_table)
        rows_of = lambda: CH.to_f64(k)[order].reshape(B, -1, H, 128)[:, :n].transpose(0, 2, 1, 3)   # noqa: E731
    else:
        k = CH.to_gpu_bf16(np.concatenate([x, np.zeros((B, H, n, 8))], -1))[..., :128]
        kv = lib().make_kv_contiguous(k, k)
        rows_of = lambda: CH.to_f64(k)   # noqa: E731
    out, ws = CH.to_gpu_bf16(np.full((B, H, n, 128), 7.0)), CH.workspace(1 << 17)
    lib().kvsel_rope_cache(t, kv, SH.ints(lens), SH.ints(pos), ws, out=out)
    assert CH.status(ws) == 0
    assert np.array_equal(rows_of(), x)
    full = lens if per_head else np.repeat(lens[:, None], H, 1)
    lib().kvsel_rope_cache(t, kv, SH.ints(lens), SH.ints(pos))
    got, here = CH.to_f64(out), rows_of()
    for b in range(B):
        for h in range(H):
            m = full[b, h]
            close(got[b, h, :m], x[b, h, :m], pos[b, h, :m], o)
            assert (got[b, h, m:] == 7.0).all()
            assert np.array_equal(here[b, h, :m], got[b, h, :m]) and np.array_equal(here[b, h, m:], x[b, h, m:])
    # the rows' own places as positions
    lib().kvsel_rope_cache(t, kv, SH.ints(lens), None, ws, out=out, batch=B, h_kv=H, max_len=n)
    for b in range(B):
        for h in range(H):
            m = full[b, h]
            close(CH.to_f64(out)[b, h, :m], here[b, h, :m], np.arange(m), o)
    # lengths and pages out of range
    lib().kvsel_rope_cache(t, kv, SH.ints(lens + 5), SH.ints(pos), ws, out=out)
    assert CH.status(ws) == -7
    if block:
        d_table[0, 0] = 10 ** 6
        lib().kvsel_rope_cache(t, kv, SH.ints(lens), SH.ints(pos), ws, out=out)
        assert CH.status(ws) == -7
    torch.cuda.synchronize()


def test_captured_and_on_other_streams():
    import torch

    t, o = table()
    g = CH.rng(3)
    x, pos = CH.bf16(g.standard_normal((2, 4, 20, 128))), g.integers(0, 1000, (2, 20))
    q, out, p = CH.to_gpu_bf16(x), CH.to_gpu_bf16(x * 0), SH.ints(pos)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            lib().kvsel_rope(t, q, p, q_out=out)
    pos = pos + 77
    p.copy_(SH.ints(pos))
    graph.replay()
    close(CH.to_f64(out), x, pos[:, None], o)
    out.zero_()
    torch.cuda.synchronize()
    lib().kvsel_rope(t, q, p, q_out=out, stream=s)
    s.synchronize()
    close(CH.to_f64(out), x, pos[:, None], o)
