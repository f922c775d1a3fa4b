"""The binding's views of caches, on CPU tensors (nothing is dereferenced): what a view cannot express is
refused when it is made."""
import pytest
import torch


@pytest.fixture(scope="module")
def B():
    import __graft_entry__

    __graft_entry__.build()
    from kv_cache_eviction_window_gb300 import binding

    binding.load()
    return binding


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def refused(B, make, *args):
    with pytest.raises(B.KvselError) as e:
        make(*args)
    assert e.value.code == B.KVSEL_EINVAL
    return True


# (k, v) as [rows][d]
PACKED_BAD = [
    (lambda: (bf16(50, 256)[:, :128], bf16(50, 128))),            # rows of k further apart
    (lambda: (bf16(50, 128), bf16(50, 256)[:, :128])),            # rows of v further apart
    (lambda: (bf16(50, 128), bf16(49, 128))),                     # fewer rows
    (lambda: (bf16(128, 50).T, bf16(128, 50).T)),                 # columns apart
    (lambda: (bf16(50, 128), bf16(128, 50).T)),
    (lambda: (bf16(50, 128), bf16(50, 128).float())),             # another type
    (lambda: (bf16(50, 128).float(), bf16(50, 128).float())),
    (lambda: (bf16(50, 128).half(), bf16(50, 128).half())),
    (lambda: (bf16(50, 128), bf16(50, 64))),                      # shorter rows
    (lambda: (bf16(128), bf16(128))),                             # no rows
]


@pytest.mark.parametrize("make", PACKED_BAD)
def test_packed_views_that_do_not_hold(B, make):
    assert refused(B, B.make_kv_packed, *make())


# (k, v) as [H][n][d] or [B][H][n][d]
CONTIGUOUS_BAD = [
    (lambda: (bf16(2, 50, 256)[..., :128], bf16(2, 50, 128))),    # rows
    (lambda: (bf16(2, 60, 128)[:, :50], bf16(2, 50, 128))),       # heads
    (lambda: (bf16(2, 50, 128), bf16(2, 60, 128)[:, :50])),
    (lambda: (bf16(3, 3, 50, 128)[:, :2], bf16(3, 2, 50, 128))),  # requests
    (lambda: (bf16(2, 50, 128), bf16(50, 2, 128).permute(1, 0, 2))),
    (lambda: (bf16(2, 128, 50).transpose(1, 2), bf16(2, 128, 50).transpose(1, 2))),
    (lambda: (bf16(2, 50, 128), bf16(1, 50, 128))),               # fewer heads
    (lambda: (bf16(2, 50, 128), bf16(2, 50, 128).float())),
    (lambda: (bf16(2, 50, 128).float(), bf16(2, 50, 128).float())),
    (lambda: (bf16(50, 128), bf16(50, 128))),
]


@pytest.mark.parametrize("make", CONTIGUOUS_BAD)
def test_contiguous_views_that_do_not_hold(B, make):
    assert refused(B, B.make_kv_contiguous, *make())


def table(*shape):
    return torch.zeros(shape, dtype=torch.int32)


# (k_pool, v_pool, block_table) as [blocks][block][H][d] twice, [B][max_blocks]
PAGED_BAD = [
    (lambda: (*bf16(7, 2, 16, 2, 128).unbind(1), table(1, 7))),               # K and V interleaved
    (lambda: (bf16(7, 16, 2, 128), bf16(7, 2, 16, 128).transpose(1, 2), table(1, 7))),
    (lambda: (bf16(7, 16, 2, 128), bf16(6, 16, 2, 128), table(1, 7))),        # fewer blocks
    (lambda: (bf16(7, 16, 2, 128), bf16(14, 8, 2, 128), table(1, 7))),        # other blocks
    (lambda: (bf16(7, 16, 2, 128), bf16(7, 16, 2, 128).float(), table(1, 7))),
    (lambda: (bf16(7, 16, 2, 128), bf16(7, 16, 2, 128), table(1, 7).long())),
    (lambda: (bf16(7, 16, 2, 128), bf16(7, 16, 2, 128), table(1, 7).float())),
    (lambda: (bf16(7, 16, 2, 128), bf16(7, 16, 2, 128), table(3, 9)[:, :7])),  # rows of the table apart
    (lambda: (bf16(7, 16, 2, 128), bf16(7, 16, 2, 128), table(7, 3).T)),
    (lambda: (bf16(7, 16, 2, 128), bf16(7, 16, 2, 128), table(7))),
]


@pytest.mark.parametrize("make", PAGED_BAD)
def test_paged_views_that_do_not_hold(B, make):
    assert refused(B, B.make_kv_paged, *make())


def test_views_that_hold(B):
    # packed: the same stride of both, one row, bit patterns in 16-bit integers
    wide = bf16(50, 2, 128)
    kv = B.make_kv_packed(wide[:, 0], wide[:, 1])
    assert (kv.stride_tok, kv.v - kv.k) == (256, 256)
    assert B.make_kv_packed(bf16(1, 256)[:, :128], bf16(1, 128)).stride_tok == 256
    assert B.make_kv_packed(bf16(5, 128).view(torch.int16), bf16(5, 128).view(torch.int16)).stride_tok == 128
    # contiguous: token-major rows, slack between heads, one request with and without its dimension
    kv = B.make_kv_contiguous(bf16(50, 4, 128).permute(1, 0, 2), bf16(50, 4, 128).permute(1, 0, 2))
    assert (kv.stride_tok, kv.stride_head) == (512, 128)
    kv = B.make_kv_contiguous(bf16(3, 2, 60, 136)[:, :, :50, :128], bf16(3, 2, 60, 136)[:, :, :55, :128])
    assert (kv.stride_tok, kv.stride_head, kv.stride_req) == (136, 60 * 136, 2 * 60 * 136)
    kv = B.make_kv_contiguous(bf16(1, 2, 50, 128), bf16(2, 50, 128))
    assert (kv.stride_tok, kv.stride_head) == (128, 6400)
    # one head: its stride does not matter; no V where a call reads none
    B.make_kv_contiguous(bf16(1, 60, 128)[:, :50], bf16(1, 50, 128))
    assert B.make_kv_contiguous(bf16(2, 50, 128), None).v is None
    assert B.make_kv_contiguous(bf16(2, 50, 128), 1 << 20).v == 1 << 20
    # paged: a slice of a longer table of one request
    kv = B.make_kv_paged(bf16(7, 16, 2, 128), bf16(9, 16, 2, 128), table(3, 9)[1:2, :7])
    assert (kv.block_size, kv.max_blocks, kv.num_blocks) == (16, 7, 7)
