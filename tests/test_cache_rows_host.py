"""Tensors of query, result and new rows that the binding's cache calls are given, on the CPU: what their
parameters do not describe is refused before anything is launched."""
import pytest
import torch


class Reached(Exception):
    """the call went on to its launch"""


@pytest.fixture
def B(monkeypatch):
    import __graft_entry__

    __graft_entry__.build()
    from kv_cache_eviction_window_gb300 import binding

    binding.load()

    def place(*a):
        raise Reached

    monkeypatch.setattr(binding, "_place", place)
    return binding


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def wide(b, m, heads, slack=2):
    """[b][heads][m][d], a slice of token-major rows with `slack` more heads."""
    return bf16(b, m, heads + slack, 128)[:, :, :heads].permute(0, 2, 1, 3)


def attend(B, q, out, q_strides=(0, 0, 0), o_strides=(0, 0, 0), b=2, m=3):
    p = B.make_attn_params(h_kv=2, group=4, batch=b, n_new=m, max_len=100, q_strides=q_strides, o_strides=o_strides)
    B.kvsel_attend(p, q, B.make_kv_contiguous(bf16(b, 2, 100, 128), bf16(b, 2, 100, 128)), None, out,
                   torch.zeros(16, dtype=torch.uint8))


def evict(B, k, v, strides=(0, 0, 0), b=2, m=3):
    p = B.make_evict_params(h_kv=2, batch=b, n_new=m, capacity=100, budget=100, new_strides=strides)
    B.kvsel_evict_append(p, B.make_kv_contiguous(bf16(b, 2, 100, 128), bf16(b, 2, 100, 128)), None, None, None, None, k, v,
                         torch.zeros(16, dtype=torch.uint8))


# ([batch][heads][tokens][d], strides) that do not belong together; 2 requests, `h` heads, 3 tokens
BAD = [
    (lambda h: (wide(2, 3, h), (0, 0, 0))),                                     # not dense
    (lambda h: (bf16(2, h, 4, 128)[:, :, :3], (0, 0, 0))),
    (lambda h: (bf16(2, h, 2, 128), (0, 0, 0))),                                # fewer tokens
    (lambda h: (bf16(1, h, 3, 128), (0, 0, 0))),                                # fewer requests
    (lambda h: (bf16(2, h, 3, 128).float(), (0, 0, 0))),                        # another type
    (lambda h: (bf16(2, h, 3, 128).half(), (0, 0, 0))),
    (lambda h: (bf16(2, h, 3, 128), (4 * h * 128, 4 * 128, 128))),              # strides that pass its end
    (lambda h: (wide(2, 2, h), (3 * (h + 2) * 128, 128, (h + 2) * 128))),
    (lambda h: (wide(2, 3, h).float(), (3 * (h + 2) * 128, 128, (h + 2) * 128))),
    (lambda h: (bf16(2, h, 128, 3).transpose(2, 3), (384 * h, 384, 128))),      # columns apart
]


@pytest.mark.parametrize("make", BAD)
def test_rows_that_do_not_hold(B, make):
    q, s = make(8)
    good = bf16(2, 8, 3, 128)
    with pytest.raises(B.KvselError) as e:
        attend(B, q, good, q_strides=s)
    assert e.value.code == B.KVSEL_EINVAL
    with pytest.raises(B.KvselError):
        attend(B, good, q, o_strides=s)
    k, s = make(2)
    with pytest.raises(B.KvselError) as e:
        evict(B, k, k, strides=s)
    assert e.value.code == B.KVSEL_EINVAL


def test_new_rows_are_both_looked_at(B):
    good, bad = bf16(2, 2, 3, 128), bf16(2, 2, 4, 128)[:, :, :3]
    for pair in ((bad, good), (good, bad)):
        with pytest.raises(B.KvselError):
            evict(B, *pair)


def test_rows_that_hold(B):
    d, t = bf16(2, 8, 3, 128), wide(2, 3, 8)
    for q, qs in ((d, (0, 0, 0)), (d, d.stride()[:3]), (t, t.stride()[:3]), (t.permute(0, 2, 1, 3), t.stride()[:3]),
                  (bf16(2, 9, 3, 128)[:, :8], (27 * 128, 384, 128)), (bf16(5, 8, 3, 128), (0, 0, 0)),
                  (d.view(torch.int16), (0, 0, 0)), (d.view(48, 128), (0, 0, 0)), (1 << 20, (0, 0, 0))):
        with pytest.raises(Reached):
            attend(B, q, d, q_strides=qs)
        with pytest.raises(Reached):
            attend(B, d, q, o_strides=qs)
    # one token, one request: strides of dimensions with one entry do not matter
    one = wide(1, 1, 8)
    for s in ((0, 0, 0), one.stride()[:3], (0, 128, 0)):
        with pytest.raises(Reached):
            attend(B, one, bf16(1, 8, 1, 128), q_strides=s, b=1, m=1)
    d, t = bf16(2, 2, 3, 128), wide(2, 3, 2)
    for k, s in ((d, (0, 0, 0)), (t, t.stride()[:3])):
        with pytest.raises(Reached):
            evict(B, k, k, strides=s)
    with pytest.raises(Reached):
        evict(B, None, None, m=0)


def test_parameters_changed_between_calls_count(B):
    p = B.make_evict_params(h_kv=2, batch=2, n_new=3, capacity=100, budget=100)
    kv = B.make_kv_contiguous(bf16(2, 2, 100, 128), bf16(2, 2, 100, 128))
    t, ws = wide(2, 3, 2), torch.zeros(16, dtype=torch.uint8)

    def call():
        B.kvsel_evict_append(p, kv, None, None, None, None, t, t, ws)

    for _ in range(2):
        with pytest.raises(B.KvselError):
            call()
    p.new_stride_req, p.new_stride_head, p.new_stride_tok = t.stride()[:3]
    for _ in range(2):
        with pytest.raises(Reached):
            call()
    p.batch = 3
    with pytest.raises(B.KvselError):
        call()
