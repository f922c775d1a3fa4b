"""What the binding of a step of drafted tokens refuses before a kernel runs."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def B():
    import __graft_entry__

    __graft_entry__.build()
    from kv_cache_eviction_window_gb300 import binding

    return binding


def test_probabilities_of_other_numbers_of_nodes_or_tokens(B):
    # [batch][n_new][vocab], dense: tensors that hold as much, in rows of another length or more of them to a request
    v = B.make_verify_params(batch=2, n_new=3, vocab=10)
    y = torch.zeros((2, 3, 10))
    for good in (y, y.view(-1), y.view(6, 10), y.view(2, 30), torch.zeros((4, 3, 10)), torch.zeros(100), torch.zeros((2, 3, 12)).view(-1)[:60].view(2, 3, 10)):
        B._values(good, v, "")
    for bad in (torch.zeros((2, 4, 10)), torch.zeros((2, 3, 11)), torch.zeros((6, 11)), torch.zeros((3, 3, 20)), torch.zeros((2, 4, 12))[:, :3, :10],
                torch.zeros(59), torch.zeros((2, 10, 3)).transpose(1, 2)):
        with pytest.raises(B.KvselError):
            B._values(bad, v, "")
    # one request: nodes behind its own do no harm
    B._values(torch.zeros((1, 5, 10)), B.make_verify_params(batch=1, n_new=3, vocab=10), "")
    # with strides: nodes 12 elements apart, requests 40
    s = B.make_verify_params(batch=2, n_new=3, vocab=10, stride_req=48, stride_node=12)
    wide = torch.zeros((2, 4, 12))
    for good in (wide, wide[:, :3, :10], wide.view(-1), wide.view(8, 12)):
        B._values(good, s, "")
    for bad in (y, torch.zeros((2, 3, 12)), torch.zeros((2, 5, 12)), wide.view(16, 6)):
        with pytest.raises(B.KvselError):
            B._values(bad, s, "")


def test_lengths_of_a_fork_that_overlap(B):
    # a row may be written before another has read it
    A = 1 << 20                                      # an address that nothing dereferences: all are refused first
    for kw, most in ((dict(), 4), (dict(lens_per_head=True), 8)):
        p = B.make_pages_params(batch=4, max_blocks=8, num_blocks=20, block_size=16, h_kv=2, **kw)
        for shift in (0, 1, most - 1, -1, 1 - most):
            assert B.load().kvsel_pages_fork(p, A, A + 4096, A, A + 65536, A + 4096 + 4 * shift, A, A, 1 << 30, None) == -1, shift


def pools(layers=3, pages=6):
    """K and V of a layer side by side: each a pool with twice a layer between layers."""
    both = torch.zeros((layers, 2, pages, 8, 2, 128), dtype=torch.bfloat16)
    return both, both[:, 0], both[:, 1]


def test_pools_with_a_stride_of_layers(B):
    both, k, v = pools()
    layer = 6 * 8 * 2 * 128
    kw = dict(batch=2, max_blocks=4, num_blocks=6, block_size=8, h_kv=2, layers=3)
    p = B.make_pages_params(stride_layer=2 * layer, **kw)
    assert p.stride_layer == 2 * layer
    assert B._pool(k, p, "") == both.data_ptr() and B._pool(v, p, "") == both.data_ptr() + 2 * layer
    B._pool(both.view(-1), p, "")
    for bad in (both[:, 0].contiguous(), k[:2], k[:, :5], both[:2, 0], k.float(), both.view(-1)[:4 * layer], both[:, :, :3].reshape(3, -1)[:, :layer],
                k.transpose(2, 3), torch.zeros((3, 6, 8, 2, 128), dtype=torch.bfloat16)):
        with pytest.raises(B.KvselError):
            B._pool(bad, p, "")
    with pytest.raises(B.KvselError):
        B._pool(k, B.make_pages_params(**kw), "")           # dense parameters
    B._pool(k[:1], B.make_pages_params(**{**kw, "layers": 1}), "")
    # layers that overlap, or begin between rows of 16 bytes
    for stride, code in ((layer - 8, -1), (8, -1), (-layer, -1), (layer + 4, -1), (layer, 0), (layer + 8, 0)):
        q = B.make_pages_params(stride_layer=stride, **kw)
        if code:
            with pytest.raises(B.KvselError) as e:
                B.kvsel_pages_workspace_size(q)
            assert e.value.code == code
        else:
            assert B.kvsel_pages_workspace_size(q) == B.kvsel_pages_workspace_size(p)
    q.stride_layer = 2 * layer                               # (what was worked out for the other stride is not kept)
    B._pool(k, q, "")
