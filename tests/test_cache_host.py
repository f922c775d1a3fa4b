"""Host-side checks of kvsel_attend and kvsel_evict_append (no GPU): struct layouts, refusals
before any CUDA work, and pins of their oracle."""
import ctypes
import math
import os
import subprocess
import tempfile

import numpy as np
import pytest

from oracle import cache_oracle as CO

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    import __graft_entry__

    __graft_entry__.build()
    from kv_cache_eviction_window_gb300 import binding

    binding.load()
    return binding


def test_struct_layouts_match_the_header(B):
    fields = [("kvsel_attn_params", f[0]) for f in B.kvsel_attn_params._fields_]
    fields += [("kvsel_evict_params", f[0]) for f in B.kvsel_evict_params._fields_]
    exprs = ["sizeof(kvsel_attn_params)", "sizeof(kvsel_evict_params)"] + [f"offsetof({s}, {f})" for s, f in fields]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "kvsel.h"\nint main(void){' + \
          "".join(f'printf("%zu\\n", (size_t){e});' for e in exprs) + "return 0;}\n"
    with tempfile.TemporaryDirectory() as d:
        c = os.path.join(d, "s.c")
        open(c, "w").write(src)
        subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", os.path.join(d, "s")])
        out = [int(x) for x in subprocess.check_output([os.path.join(d, "s")]).split()]
    want = [ctypes.sizeof(B.kvsel_attn_params), ctypes.sizeof(B.kvsel_evict_params)]
    want += [getattr(getattr(B, s), f).offset for s, f in fields]
    assert out == want


GOOD = 1 << 20     # an aligned address that nothing dereferences: every case below is refused first


def attend(B, kv=None, ptr=None, ws_bytes=1 << 40, **kw):
    base = dict(h_kv=2, group=4, batch=1, max_len=100)
    base.update(kw)
    p = B.make_attn_params(**base)
    if kv is None:
        kv = contiguous(B)
    a = dict(q=GOOD, lens=GOOD, new_lens=None, offsets=None, out=GOOD, lse=None, acc=None, ws=GOOD)
    a.update(ptr or {})
    return B.load().kvsel_attend(ctypes.byref(p), a["q"], ctypes.byref(kv), a["lens"], a["new_lens"], a["offsets"], a["out"],
                                 a["lse"], a["acc"], a["ws"], ws_bytes, None)


def contiguous(B, **kw):
    kv = B.kvsel_kv()
    kv.k = kv.v = GOOD
    kv.stride_tok, kv.stride_head, kv.stride_req = 128, 12800, 25600
    for f, x in kw.items():
        setattr(kv, f, x)
    return kv


def paged(B, **kw):
    base = dict(layout=1, block_table=GOOD, block_size=16, max_blocks=7, num_blocks=7)
    base.update(kw)
    return contiguous(B, **base)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=64), -3), (dict(h_kv=0), -1), (dict(h_kv=65), -1), (dict(group=0), -1), (dict(group=129), -3),
    (dict(batch=0), -1), (dict(batch=1025), -3), (dict(n_new=0), -1), (dict(n_new=(1 << 20) + 1), -3),
    (dict(max_len=0), -1), (dict(max_len=(1 << 30) + 1), -3), (dict(window=-1), -1), (dict(n_sink=-1), -1),
    (dict(window=5, causal=False), -3), (dict(scale=-1.0), -1), (dict(scale=float("inf")), -1),
    (dict(scale=float("nan")), -1), (dict(q_strides=(0, 128, 4), n_new=2), -1), (dict(o_strides=(0, 0, 128), n_new=2), -1),
    (dict(q_strides=(-8, 128, 128), batch=2), -1), (dict(n_new=1 << 20, group=128, h_kv=64), -3),
    (dict(batch=1024, h_kv=64), -3)])
def test_attend_refuses_parameters(B, kw, code):
    assert attend(B, **kw) == code


@pytest.mark.parametrize("ptr", [dict(q=None), dict(q=GOOD + 8), dict(lens=None), dict(lens=GOOD + 2), dict(out=None),
                                 dict(out=GOOD + 4), dict(lse=GOOD + 1), dict(new_lens=GOOD + 1), dict(acc=GOOD),
                                 dict(offsets=GOOD)])
def test_attend_refuses_pointers(B, ptr):
    # (acc without an acc_stride, offsets without a packed cache)
    assert attend(B, ptr=ptr) == B.KVSEL_EINVAL


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=GOOD + 2), dict(stride_tok=64), dict(stride_tok=129),
                                dict(stride_head=0), dict(stride_head=-12800), dict(layout=3), dict(layout=2)])
def test_attend_refuses_caches(B, kw):
    assert attend(B, kv=contiguous(B, **kw)) == B.KVSEL_EINVAL


@pytest.mark.parametrize("kw", [dict(block_table=None), dict(block_size=4), dict(block_size=128), dict(max_blocks=6),
                                dict(num_blocks=0)])
def test_attend_refuses_block_tables(B, kw):
    assert attend(B, kv=paged(B, **kw)) == B.KVSEL_EINVAL


def evict(B, kv=None, ptr=None, ws_bytes=1 << 40, **kw):
    base = dict(h_kv=2, batch=1, capacity=100, budget=100)
    base.update(kw)
    p = B.make_evict_params(**base)
    a = dict(lens=GOOD, seen=GOOD, pos=GOOD, acc=GOOD, k_new=GOOD, v_new=GOOD, new_lens=None, ws=GOOD)
    a.update(ptr or {})
    kv = kv or contiguous(B)
    return B.load().kvsel_evict_append(ctypes.byref(p), ctypes.byref(kv), a["lens"], a["seen"], a["pos"], a["acc"], a["k_new"],
                                       a["v_new"], a["new_lens"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=64), -3), (dict(h_kv=0), -1), (dict(h_kv=65), -1), (dict(batch=0), -1), (dict(batch=1025), -3),
    (dict(n_new=-1), -1), (dict(capacity=0), -1), (dict(budget=0), -1), (dict(budget=101), -1), (dict(n_sink=-1), -1),
    (dict(n_recent=-1), -1), (dict(n_sink=60, n_recent=41), -2), (dict(n_new=97), -2), (dict(n_new=101, n_sink=0), -2),
    (dict(new_strides=(0, 128, 100), n_new=2), -1),
    (dict(batch=1024, h_kv=64), -3)])
def test_evict_refuses_parameters(B, kw, code):
    assert evict(B, **kw) == code
    if "new_strides" not in kw:
        with pytest.raises(B.KvselError) as e:
            B.kvsel_evict_append_workspace_size(B.make_evict_params(**{**dict(h_kv=2, batch=1, capacity=100, budget=100), **kw}))
        assert e.value.code == code


@pytest.mark.parametrize("ptr,code", [(dict(lens=None), -1), (dict(seen=None), -1), (dict(pos=None), -1), (dict(acc=None), -1),
                                      (dict(k_new=None), -1), (dict(v_new=GOOD + 8), -1), (dict(pos=GOOD + 2), -1),
                                      (dict(ws=None), -4), (dict(ws=GOOD + 16), -4)])
def test_evict_refuses_pointers(B, ptr, code):
    assert evict(B, ptr=ptr) == code


def test_evict_workspace_serves_a_cache_for_good(B):
    size = lambda **kw: B.kvsel_evict_append_workspace_size(B.make_evict_params(h_kv=8, batch=4, capacity=4096, **kw))   # noqa: E731
    assert size(budget=4096, n_new=1) == size(budget=100, n_new=50) == size(budget=4000, n_new=0)


def test_evict_refuses_caches_and_small_workspaces(B):
    assert evict(B, kv=contiguous(B, layout=2)) == B.KVSEL_EINVAL          # packed rows have no room to grow
    assert evict(B, kv=paged(B, max_blocks=6)) == B.KVSEL_EINVAL
    need = B.kvsel_evict_append_workspace_size(B.make_evict_params(h_kv=2, batch=1, capacity=100, budget=100))
    assert evict(B, ws_bytes=need - 1) == B.KVSEL_EWORKSPACE


# ------------------------------------------------------------------------------ oracle pins
def test_oracle_attention_by_hand():
    # three rows with logits 0, ln 2, ln 3 for a unit query: weights 1/6, 2/6, 3/6
    d = 128
    q, k, v = np.zeros((1, 1, d)), np.zeros((3, d)), np.zeros((3, d))
    q[0, 0, 0] = 1.0
    k[:, 0] = np.log([1.0, 2.0, 3.0]) * math.sqrt(d)
    v[:, 1] = [6.0, 12.0, 24.0]
    o = CO.attend_segment(q, k, v)
    assert np.allclose(o["out"][0, 0, 1], 1 + 4 + 12) and np.allclose(o["lse"], math.log(6.0))
    assert np.allclose(o["weight"], [1 / 6, 2 / 6, 3 / 6])


def test_oracle_visibility_by_hand():
    # rows 0..5, two new tokens at rows 4 and 5; window 2 with one first token
    see = CO.visible(6, 2, True, 2, 1)
    assert see.astype(int).tolist() == [[1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert CO.visible(1, 3, True, 0, 0).astype(int).tolist() == [[0], [0], [1]]
    assert CO.visible(2, 1, False, 0, 0).all()


def test_oracle_eviction_by_hand():
    # 6 rows, one new token, budget 5: 4 stay.  Position 0 is protected, so is position 9 (the most
    # recent); of the others the two largest stay (0.7, then the first of the tied 0.5s)
    pos, acc = np.array([0, 3, 4, 5, 8, 9]), np.array([0.0, 0.1, 0.5, 0.7, 0.5, 0.0])
    # rows 0, 2, 3, 5 stay: hole 1 takes row 5
    assert CO.evict_segment(pos, acc, 10, 1, budget=5, n_sink=1, n_recent=2) == [0, 5, 2, 3]
    # nothing to do while there is room
    assert CO.evict_segment(pos, acc, 10, 1, budget=7, n_sink=1, n_recent=2) == [0, 1, 2, 3, 4, 5]
    # NaN leaves first
    assert CO.evict_segment(pos, np.array([0, np.nan, -1.0, 0.7, 0.5, 0]), 10, 1, budget=6, n_sink=1, n_recent=2) == [0, 5, 2, 3, 4]
