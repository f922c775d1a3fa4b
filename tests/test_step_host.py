"""Host-side checks of a step of drafted tokens (no GPU): struct layouts, refusals before any CUDA work,
the angles of rotary positions, and pins of the oracle."""
import ctypes
import math
import os
import subprocess
import tempfile
from fractions import Fraction

import numpy as np
import pytest

from oracle import step_oracle as SO

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = 1 << 20     # an aligned address that nothing dereferences: every case below is refused first
WS = 1 << 40


@pytest.fixture(scope="module")
def B():
    import __graft_entry__

    __graft_entry__.build()
    from kv_cache_eviction_window_gb300 import binding

    binding.load()
    return binding


def test_struct_layouts_match_the_header(B):
    names = ["kvsel_verify_params", "kvsel_pages_params", "kvsel_rope_params", "kvsel_rope_angles", "kvsel_rope_rows",
             "kvsel_rope_cache_params"]
    fields = [(s, f[0]) for s in names for f in getattr(B, s)._fields_]
    exprs = [f"sizeof({s})" for s in names] + [f"offsetof({s}, {f})" for s, f in fields]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "kvsel.h"\nint main(void){' + \
          "".join(f'printf("%zu\\n", (size_t){e});' for e in exprs) + "return 0;}\n"
    with tempfile.TemporaryDirectory() as d:
        c = os.path.join(d, "s.c")
        open(c, "w").write(src)
        subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", os.path.join(d, "s")])
        out = [int(x) for x in subprocess.check_output([os.path.join(d, "s")]).split()]
    assert out == [ctypes.sizeof(getattr(B, s)) for s in names] + [getattr(getattr(B, s), f).offset for s, f in fields]


# ------------------------------------------------------------------------------ refusals
def contiguous(B, **kw):
    kv = B.kvsel_kv()
    kv.k = kv.v = GOOD
    kv.stride_tok, kv.stride_head, kv.stride_req = 128, 12800, 25600
    for f, x in kw.items():
        setattr(kv, f, x)
    return kv


def tree(B, kv=None, ws_bytes=WS, ptr=None, **kw):
    p = B.make_attn_params(**dict(dict(h_kv=2, group=4, batch=1, max_len=100, n_new=8), **kw))
    a = dict(dict(q=GOOD, lens=GOOD, new_lens=None, offsets=None, tree=GOOD, out=GOOD, lse=None, ws=GOOD), **(ptr or {}))
    return B.load().kvsel_attend_tree(p, a["q"], kv or contiguous(B), a["lens"], a["new_lens"], a["offsets"], a["tree"], a["out"],
                                      a["lse"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("kw,code", [(dict(n_new=1025), -3), (dict(causal=False), -3), (dict(n_new=0), -1), (dict(head_dim=64), -3),
                                     (dict(window=-1), -1), (dict(group=129), -3), (dict(scale=float("nan")), -1)])
def test_tree_refuses_parameters(B, kw, code):
    assert tree(B, **kw) == code
    with pytest.raises(B.KvselError) as e:
        B.kvsel_attend_tree_workspace_size(B.make_attn_params(**dict(dict(h_kv=2, group=4, batch=1, max_len=100, n_new=8), **kw)))
    assert e.value.code == code


@pytest.mark.parametrize("ptr", [dict(tree=None), dict(tree=GOOD + 2), dict(q=None), dict(lens=None), dict(out=GOOD + 8),
                                 dict(lse=GOOD + 2), dict(new_lens=GOOD + 1), dict(offsets=GOOD)])
def test_tree_refuses_pointers(B, ptr):
    assert tree(B, ptr=ptr) == B.KVSEL_EINVAL


def masks(B, parents=GOOD, new_lens=None, first=GOOD, batch=1, n_new=8, tree=GOOD, pos=GOOD):
    return B.load().kvsel_tree_masks(parents, new_lens, first, batch, n_new, tree, pos, None)


@pytest.mark.parametrize("kw,code", [(dict(parents=None), -1), (dict(tree=None), -1), (dict(first=None), -1), (dict(pos=GOOD + 2), -1),
                                     (dict(new_lens=GOOD + 1), -1), (dict(batch=0), -1), (dict(n_new=0), -1), (dict(batch=1025), -3),
                                     (dict(n_new=1025), -3)])
def test_masks_refuse(B, kw, code):
    assert masks(B, **kw) == code


def verify(B, ptr=None, ws_bytes=WS, **kw):
    p = B.make_verify_params(**dict(dict(batch=2, n_new=8, vocab=100), **kw))
    a = dict(dict(tokens=GOOD, parents=GOOD, target=GOOD, draft=GOOD, u=GOOD, new_lens=None, path=GOOD, counts=GOOD, next=GOOD, ws=GOOD),
             **(ptr or {}))
    return B.load().kvsel_verify(p, a["tokens"], a["parents"], a["target"], a["draft"], a["u"], a["new_lens"], a["path"], a["counts"],
                                 a["next"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("kw,code", [(dict(batch=0), -1), (dict(batch=1025), -3), (dict(n_new=0), -1), (dict(n_new=1025), -3),
                                     (dict(vocab=0), -1), (dict(vocab=262145), -3), (dict(stride_node=99, stride_req=5000), -1),
                                     (dict(stride_node=100, stride_req=99), -1)])
def test_verify_refuses_parameters(B, kw, code):
    assert verify(B, **kw) == code


@pytest.mark.parametrize("ptr,code", [({x: None}, -1) for x in ("tokens", "parents", "target", "draft", "u", "path", "counts", "next")] + [
    (dict(target=GOOD + 2), -1), (dict(draft=GOOD + 1), -1), (dict(ws=None), -4), (dict(ws=GOOD + 16), -4)])
def test_verify_refuses_pointers(B, ptr, code):
    assert verify(B, ptr=ptr) == code


def test_verify_refuses_what_a_mode_does_not_take(B):
    assert verify(B, mode="point") == -1 and verify(B, mode="greedy") == -1          # a draft
    assert verify(B, mode="point", ptr=dict(draft=None, u=None)) == -1
    assert verify(B, ws_bytes=255) == -4
    p = B.make_verify_params(batch=2, n_new=8, vocab=100)
    for f, x in (("mode", 3), ("dtype", 2), ("mode", -1)):
        q = B.make_verify_params(batch=2, n_new=8, vocab=100)
        setattr(q, f, x)
        with pytest.raises(B.KvselError):
            B.kvsel_verify_workspace_size(q)
    assert B.kvsel_verify_workspace_size(p) == 256


PAGES = dict(batch=2, max_blocks=8, num_blocks=30, block_size=16, h_kv=2)


@pytest.mark.parametrize("kw,code", [(dict(batch=0), -1), (dict(batch=1025), -3), (dict(max_blocks=0), -1), (dict(max_blocks=(1 << 20) + 1), -3),
                                     (dict(num_blocks=0), -1), (dict(num_blocks=(1 << 28) + 1), -3), (dict(block_size=12), -1),
                                     (dict(h_kv=65), -1), (dict(layers=0), -1), (dict(layers=1025), -3), (dict(n_new=-1), -1),
                                     (dict(head_dim=64), -3), (dict(n_new=(1 << 20) + 1), -3), (dict(n_new=1 << 20, batch=64), -3)])
def test_pages_refuse_parameters(B, kw, code):
    with pytest.raises(B.KvselError) as e:
        B.kvsel_pages_workspace_size(B.make_pages_params(**{**PAGES, **kw}))
    assert e.value.code == code


def test_pages_refuse_pointers(B):
    lib, p = B.load(), B.make_pages_params(**PAGES)
    size = B.kvsel_pages_workspace_size(p)
    G2 = GOOD + (1 << 16)
    calls = {"fork": (lib.kvsel_pages_fork, [GOOD, GOOD, GOOD, G2, G2, GOOD]),
             "reserve": (lib.kvsel_pages_reserve, [GOOD, GOOD, GOOD, GOOD, GOOD, None, GOOD]),
             "trim": (lib.kvsel_pages_trim, [GOOD, GOOD, GOOD]),
             "accept": (lib.kvsel_pages_accept, [GOOD, GOOD, GOOD, GOOD, None, GOOD, GOOD, GOOD])}
    for name, (f, args) in calls.items():
        for i, x in enumerate(args):
            for bad in ([None] if x is not None else []) + [GOOD + 2]:
                assert f(p, *args[:i], bad, *args[i + 1:], GOOD, WS, None) == -1, (name, i)
        assert f(p, *args, None, WS, None) == -4 and f(p, *args, GOOD, size - 1, None) == -4 and f(p, *args, GOOD + 8, WS, None) == -4
    # rows that overlap
    assert lib.kvsel_pages_fork(p, GOOD, GOOD, GOOD, GOOD + 60, G2, GOOD, GOOD, WS, None) == -1
    assert lib.kvsel_pages_fork(p, GOOD, GOOD, GOOD, G2, GOOD, GOOD, GOOD, WS, None) == -1
    q = B.make_pages_params(**{**PAGES, "n_new": 0})
    assert lib.kvsel_pages_accept(q, *calls["accept"][1], GOOD, WS, None) == -1


def keep(B, kv=None, capacity=100, ws=None, ws_bytes=0, **ptr):
    p = B.make_params(h_kv=2, group=1, n_ctx=100, window=32, n_sink=0, n_recent=0)
    a = dict(dict(idx=GOOD, counts=GOOD, offsets=GOOD, scores=None, lens=GOOD, seen=None, pos=GOOD, acc=None), **ptr)
    return B.load().kvsel_compact_in_place(p, kv or contiguous(B), a["idx"], a["counts"], a["offsets"], a["scores"], a["lens"], a["seen"],
                                           a["pos"], a["acc"], capacity, ws, ws_bytes, None)


def test_keep_refuses(B):
    for name in ("idx", "counts", "offsets", "lens", "pos"):
        assert keep(B, **{name: None}) == -1
    for name in ("idx", "offsets", "scores", "seen", "acc"):
        assert keep(B, **{name: GOOD + 2}) == -1
    assert keep(B, offsets=GOOD + 4) == -1 and keep(B, capacity=99) == -1
    assert keep(B, kv=contiguous(B, layout=2)) == -1 and keep(B, kv=contiguous(B, v=None)) == -1
    assert keep(B, ws=GOOD, ws_bytes=255) == -4 and keep(B, ws=GOOD + 4, ws_bytes=WS) == -4


def test_rope_refuses(B):
    for kw, code in ((dict(rot_dim=0), -1), (dict(rot_dim=24), -3), (dict(rot_dim=144), -3), (dict(rot_dim=16, scaling="ntk"), -3),
                     (dict(theta=1.0), -1), (dict(theta=float("inf")), -1), (dict(scaling="linear", factor=0.5), -1),
                     (dict(scaling="yarn", factor=2.0), -1), (dict(scaling="bands", factor=2.0), -1), (dict(value_scale=-1.0), -1),
                     (dict(scaling="yarn", factor=2.0, orig_len=100, beta_fast=1.0), -1),
                     (dict(scaling="bands", factor=2.0, orig_len=100, low_freq=4.0), -1),
                     (dict(scaling="linear", factor=float("nan")), -1)):
        with pytest.raises(B.KvselError) as e:
            B.kvsel_rope_table(**kw)
        assert e.value.code == code, kw
    t = B.kvsel_rope_table()
    rows = dict(batch=2, n_tok=3, heads=4, k_heads=1, q_req=1536, q_head=384, q_tok=128, qo_req=1536, qo_head=384, qo_tok=128,
                k_req=384, k_head=384, k_tok=128, ko_req=384, ko_head=384, ko_tok=128, pos_req=3)

    def call(table=t, q=GOOD, qo=GOOD, k=GOOD, ko=GOOD, pos=GOOD, new_lens=None, **kw):
        return B.load().kvsel_rope(table, B.kvsel_rope_rows(**{**rows, **kw}), q, qo, k, ko, pos, new_lens, None)

    for kw, code in ((dict(q=None), -1), (dict(qo=GOOD + 8), -1), (dict(k=None), -1), (dict(ko=GOOD + 2), -1), (dict(pos=None), -1),
                     (dict(pos=GOOD + 2), -1), (dict(new_lens=GOOD + 1), -1), (dict(batch=0), -1), (dict(batch=65536), -3),
                     (dict(n_tok=0), -1), (dict(n_tok=(1 << 20) + 1), -3), (dict(heads=0), -1), (dict(heads=8192), -3), (dict(k_heads=-1), -1),
                     (dict(q_tok=100), -1), (dict(qo_head=0), -1), (dict(ko_req=-8), -1), (dict(pos_req=-1), -1)):
        assert call(**kw) == code, kw
    # in place, but not to the same rows
    for kw in (dict(qo_req=4608), dict(qo_tok=512, qo_head=128), dict(ko_tok=256), dict(ko_req=768)):
        assert call(**kw) == -1, kw
    bad = B.kvsel_rope_table()
    bad.rot_dim = 130
    assert call(table=bad) == -1
    cache = dict(h_kv=2, batch=1, max_len=100, lens_per_head=0, pos_stride=100, o_req=25600, o_head=12800, o_tok=128)

    def turn(kv=None, lens=GOOD, pos=GOOD, out=None, ws=None, ws_bytes=0, **kw):
        return B.load().kvsel_rope_cache(t, B.kvsel_rope_cache_params(**{**cache, **kw}), kv or contiguous(B), lens, pos, out, ws, ws_bytes, None)

    for kw, code in ((dict(lens=None), -1), (dict(pos=None), -1), (dict(pos_stride=0), -1), (dict(pos_stride=99), -1), (dict(max_len=0), -1),
                     (dict(h_kv=65), -1), (dict(batch=1025), -3), (dict(max_len=(1 << 30) + 1), -3), (dict(out=GOOD, o_tok=4), -1),
                     (dict(out=GOOD + 2), -1), (dict(ws=GOOD, ws_bytes=100), -4), (dict(kv=contiguous(B, layout=2)), -1),
                     (dict(kv=contiguous(B, stride_tok=64)), -1), (dict(kv=contiguous(B, layout=1)), -1)):
        assert turn(**kw) == code, kw


def test_binding_refuses_tensors_of_other_shapes(B):
    import torch

    t = B.kvsel_rope_table()
    x, pos = torch.zeros((2, 3, 5, 128), dtype=torch.bfloat16), torch.zeros((2, 5), dtype=torch.int32)
    for kw in (dict(q=x.float()), dict(q=x[..., :64]), dict(pos=pos.long()), dict(pos=pos[:, :4]), dict(k=x[:1]), dict(q_out=x[:, :2]),
               dict(q=x.transpose(2, 3)), dict(pos=pos.t())):
        with pytest.raises(B.KvselError):
            B.kvsel_rope(t, **dict(dict(q=x, pos=pos), **kw))
    p = B.make_pages_params(batch=2, max_blocks=4, num_blocks=6, block_size=8, h_kv=2, layers=2)
    k = torch.zeros((2, 6, 8, 2, 128), dtype=torch.bfloat16)
    for bad in (k[:1], k.float(), k.transpose(1, 2)):
        with pytest.raises(B.KvselError):
            B._pool(bad, p, "")
    i = torch.zeros(8, dtype=torch.int32)
    for bad in (i.float(), i.long(), i[::2], i[:7]):
        with pytest.raises(B.KvselError):
            B._int32(bad, 8, "")
    v = B.make_verify_params(batch=2, n_new=3, vocab=10)
    y = torch.zeros((2, 3, 10))
    for bad in (y.double(), y.bfloat16(), y[:, :2], y[..., :9], torch.zeros((2, 3, 12))[..., :10]):
        with pytest.raises(B.KvselError):
            B._values(bad, v, "")


# ------------------------------------------------------------------------------ angles
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 3.0), ("ntk", 5.0), ("yarn", 16.0), ("yarn", 1.0), ("bands", 8.0)])
@pytest.mark.parametrize("rot", [32, 64, 128])
def test_angles(B, scaling, factor, rot):
    t = B.kvsel_rope_table(rot_dim=rot, theta=500000.0, scaling=scaling, factor=factor, orig_len=8192)
    f, scale = SO.frequencies(rot, 500000.0, scaling, factor, 8192)
    got = np.array([t.turns[i] for i in range(rot // 2)], np.float64) / 2.0 ** 64 * 2 * math.pi
    # two ways to the same number in 64 bits: powers and logarithms of a few roundings each; the table is cut to
    # whole units of 2^-64 turns, which is 2 pi 2^-64 = 3.4e-19 radians: 2e-13 of a frequency of 1.5e-6
    assert np.allclose(got, f, rtol=1e-13, atol=2 * math.pi * 2.0 ** -64) and abs(t.scale - scale) <= 2.0 ** -24 * scale
    assert all(t.turns[i] == 0 for i in range(rot // 2, 64))
    assert t.rot_dim == rot and t.back == 0
    inv = B.kvsel_rope_table(rot_dim=rot, theta=500000.0, scaling=scaling, factor=factor, orig_len=8192, direction="inverse")
    assert inv.back == 1 and abs(inv.scale * scale - 1) <= 2.0 ** -23
    tr = B.kvsel_rope_table(rot_dim=rot, scaling=scaling, factor=factor, orig_len=8192, direction="transpose", value_scale=3.0)
    assert tr.back == 1 and tr.scale == 3.0


# ------------------------------------------------------------------------------ oracle pins
def test_oracle_tree_by_hand():
    see = SO.ancestors([-1, 0, 0, 1, 2])
    assert see.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 1, 0, 1, 0], [1, 0, 1, 0, 1]]
    assert SO.words(see, 5).ravel().tolist() == [1, 3, 5, 11, 21]
    # seven rows, the last five the tree's; window 2: node 1 (row 3) sees row 2, node 3 (row 4) none before
    vis = SO.tree_visible(7, see, 2, 0)
    assert vis[:, :2].astype(int).tolist() == [[0, 1], [0, 0], [0, 0], [0, 0], [0, 0]]
    assert SO.tree_visible(7, see, 2, 1)[3].astype(int).tolist() == [1, 0, 1, 1, 0, 1, 0]
    # a chain is causal (where the window does not end inside the tree, whose rows the masks alone decide)
    from oracle import cache_oracle as CO

    chain = SO.ancestors([t - 1 for t in range(6)])
    for n, window, sink in ((20, 0, 0), (20, 7, 2), (6, 6, 0)):
        assert np.array_equal(SO.tree_visible(n, chain, window, sink), CO.visible(n, 6, True, window, sink))


def test_oracle_verification_by_hand():
    p, q = [[0.5, 0.25, 0.25], [0.0, 1.0, 0.0]], [[0.25, 0.5, 0.25], [1 / 3] * 3]
    # token 1: accepted below 0.25 / 0.5; then the draw from p_1
    assert SO.verify([9, 1], [-1, 0], p, q, [0.9, 0.4999], "sampled") == ([0, 1], 1)
    # rejected: what is left of p - q is at token 0 alone
    assert SO.verify([9, 1], [-1, 0], p, q, [0.9, 0.5], "sampled") == ([0], 0)
    # point: 0.25 of the target; then 0.5, 0, 0.25: token 2 from two thirds on
    assert SO.verify([9, 1], [-1, 0], p, None, [0.6, 0.25], "point") == ([0], 0)
    assert SO.verify([9, 1], [-1, 0], p, None, [0.7, 0.25], "point") == ([0], 2)
    # a second child after a rejection: 0.25 of the 0.75 that is left
    assert SO.verify([9, 1, 2], [-1, 0, 0], p + p, None, [0.0, 0.3, 0.33], "point")[0] == [0, 2]
    assert SO.verify([9, 1, 2], [-1, 0, 0], p + p, None, [0.0, 0.3, 0.34], "point")[0] == [0]
    assert SO.verify([9, 1, 0], [-1, 0, 0], p + p, None, [0, 0], "greedy") == ([0, 2], 0)
    assert SO.verify([], [], [], None, [], "greedy") == ([], -1)


@pytest.mark.parametrize("kids", [1, 2, 3])
def test_oracle_follows_the_target(kids):
    # the first token's exact distribution over all drafts and a grid of random numbers, three tokens
    p, q = [Fraction(1, 2), Fraction(3, 8), Fraction(1, 8)], [Fraction(1, 4), Fraction(1, 4), Fraction(1, 2)]
    rows = [[float(x) for x in p]] * (kids + 1)
    drafts = [[float(x) for x in q]] * (kids + 1)
    total = [Fraction(0)] * 3

    def walk(t, tokens, us, weight):
        if t > kids:
            for cell in range(48):
                path, nxt = SO.verify([0] + tokens, [-1] + [0] * kids, rows, drafts, [(cell + 0.5) / 48] + us, "sampled")
                total[tokens[path[1] - 1] if len(path) > 1 else nxt] += weight / 48
            return
        for x in range(3):
            # u in the middle of 16 cells (and u_0 of 48): the borders, 1/4 and 2/3, lie between cells
            for cell in range(16):
                walk(t + 1, tokens + [x], us + [(cell + 0.5) / 16], weight * q[x] / 16)

    if kids <= 1:
        walk(1, [], [], Fraction(1))
        assert total == p
    else:
        # by the formula: accepted mass and what is left, child after child
        r, Z, got, alive = list(p), Fraction(1), [Fraction(0)] * 3, Fraction(1)
        for _ in range(kids):
            for x in range(3):
                got[x] += alive * min(q[x], r[x] / Z)
            alive *= 1 - sum(min(q[x], r[x] / Z) for x in range(3))
            r = [max(a - Z * b, Fraction(0)) for a, b in zip(r, q)]
            Z = sum(r)
        got = [a + alive * b / Z for a, b in zip(got, r)]
        assert got == p


def test_oracle_pages_by_hand():
    k = np.arange(6)[None, :, None, None, None] * np.ones((1, 6, 8, 1, 1))
    o = SO.Pages(np.array([[4, -1, -1], [4, -1, -1]]), np.array([0, 1, 0, 0, 2, 0]), k, k)
    # both write to page 4: the first gets a copy of its rows, the second keeps it; then a page each
    assert o.reserve([5, 5], [4, 1]).tolist() == [4, 1]
    assert o.table.tolist() == [[0, 2, -1], [4, -1, -1]] and o.ref.tolist() == [1, 1, 1, 0, 1, 0]
    assert o.k[0, 0, :, 0, 0].tolist() == [4] * 5 + [0] * 3
    o.fork([1, 1])
    assert o.table.tolist() == [[4, -1, -1]] * 2 and o.ref.tolist() == [0, 1, 0, 0, 2, 0]
    o.trim([0, 8])
    assert o.ref.tolist() == [0, 1, 0, 0, 1, 0]
    # no page is left: request 0 stays on the page, so request 1 cannot have it for itself
    o = SO.Pages(np.array([[0, -1], [0, -1]]), np.array([2]), k[:, :1], k[:, :1])
    assert o.reserve([5, 3], [1, 1]).tolist() == [0, 0] and o.table.tolist() == [[0, -1]] * 2 and o.ref.tolist() == [2]
    assert SO.keep_rows(6, [0, 3, 5]) == [0, 3, 5] and SO.keep_rows(6, [1, 2, 4]) == [4, 1, 2]


def test_oracle_rope_by_hand():
    x = np.zeros(128)
    x[0], x[64], x[1], x[127] = 1.0, 2.0, 3.0, 5.0
    f = np.zeros(64)
    f[0] = math.pi / 2
    y = SO.rope(x, 1, f)
    assert np.allclose(y[[0, 64]], [-2.0, 1.0]) and y[1] == 3.0 and y[127] == 5.0
    y = SO.rope(x, 1, f, interleaved=True)
    assert np.allclose(y[[0, 1]], [-3.0, 1.0]) and y[64] == 2.0
    assert np.allclose(SO.rope(SO.rope(x, 3, f + 0.1, 1.7), 3, f + 0.1, 1.7, direction="inverse"), x)
