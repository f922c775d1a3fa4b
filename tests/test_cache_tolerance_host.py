"""That the bounds of the tests on the GPU can tell what they are there for, on the CPU: the second product
of the kernel of few rows restated with and without the weights' remainder, and with rows left out."""
import numpy as np
import pytest

from tests import cache_harness as CH


def restated(c, b, h, remainder=True, skip=None):
    """Results of one segment from bf16 parts of the weights, rounded to bf16; rows in `skip` are lost."""
    k, v, q = c.k[b][h], c.v[b][h].copy(), c.q[b, h]
    n, m = k.shape[0], c.new[b]
    if skip is not None:
        v[skip] = 0.0
    out = np.zeros((c.G, m, CH.D))
    for g in range(c.G):
        for t in range(m):
            see = n - m + t + 1
            y = k[:see] @ q[g, t] * (c.scale or CH.D ** -0.5)
            p = np.exp(y - y.max()).astype(np.float32).astype(np.float64)
            hi = CH.bf16(p)
            w = hi + CH.bf16(p - hi) if remainder else hi
            out[g, t] = CH.bf16(w @ v[:see] / p.sum())
    return out


@pytest.mark.parametrize("n", [2, 3, 7, 16, 40, 64])
def test_a_missing_remainder_shows(n):
    c = CH.paired(CH.Case(H=1, G=8, lens=n, logit=0.1, seed=n))
    o = c.oracle()[0][0]
    tol = CH.token_tolerance(o, n)
    assert np.all(np.abs(restated(c, 0, 0) - o["out"]) <= tol)
    assert np.any(np.abs(restated(c, 0, 0, remainder=False) - o["out"]) > tol)


@pytest.mark.parametrize("G,m,n", [(8, 1, 20011), (5, 4, 12000), (2, 1, 700)])
def test_lost_rows_show(G, m, n):
    c = CH.marked(CH.Case(H=1, G=G, m=m, lens=n, scale=1e-3, seed=n))
    o = c.oracle()[0][0]
    # the wider bound, of weights rounded to bf16
    e = (CH.D + 4) * 2.0 ** -23 * o["abs_logit"] + 2.0 ** -14
    tol = (2 * e[..., None] + 2.0 ** -8) * o["mean_abs"] + 2.0 ** -8 * np.abs(o["out"]) + 1e-30
    assert np.all(np.abs(restated(c, 0, 0, remainder=False) - o["out"]) <= tol)
    for j in list(range(0, n - 16, 16 * 37)) + [(n - 1) // 16 * 16 - 16]:
        err = np.abs(restated(c, 0, 0, skip=slice(j, j + 16)) - o["out"])
        assert np.all((err > tol).any(axis=-1)), j
