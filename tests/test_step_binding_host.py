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
