"""fp64 CPU oracle for the calls that use a compacted cache: attention of new tokens with the
running weight of every cached row, and eviction by that weight.

TEST INFRASTRUCTURE ONLY (see oracle/kvsel_oracle.py): plain restatements of the definitions
with numpy steps, one segment at a time, sharing no code with the CUDA library.

Definitions: attention over the cached rows is the softmax-weighted sum of the value rows (GQA: the
group's query heads share a segment); accumulated attention weight of a cached row is the
sum of its softmax weights over the new tokens and the group; eviction keeps the protected
positions first, then the rows with the largest accumulated weight.
"""
from __future__ import annotations

import math
from typing import Optional

import numpy as np


def visible(n: int, m: int, causal: bool, window: int, n_sink: int) -> np.ndarray:
    """[m][n]: whether new token t (row n - m + t) sees row j."""
    r = n - m + np.arange(m)[:, None]
    j = np.arange(n)[None, :]
    if not causal:
        return np.ones((m, n), bool)
    see = j <= r
    if window:
        see &= (j > r - window) | (j < n_sink)
    return see


def attend_segment(q: np.ndarray, k: np.ndarray, v: np.ndarray, *, causal: bool = True, window: int = 0,
                   n_sink: int = 0, scale: Optional[float] = None) -> dict:
    """q [G][m][d], k and v [n][d] (float64).  out [G][m][d], lse [G][m], weight [n], and
    mean_abs [G][m][d] = sum_j w_j |v_j|, abs_logit [G][m] = max_j scale * sum |q||k| over the
    visible rows (what rounding errors scale with)."""
    G, m, d = q.shape
    n = k.shape[0]
    s = scale or 1.0 / math.sqrt(d)
    see = visible(n, m, causal, window, n_sink)
    any_row = see.any(axis=0)
    k = np.where(any_row[:, None], k, 0.0)      # rows that no token sees may hold anything
    v = np.where(any_row[:, None], v, 0.0)
    out, mean_abs = np.zeros((G, m, d)), np.zeros((G, m, d))
    lse = np.full((G, m), -np.inf)
    size = np.zeros((G, m))
    weight = np.zeros(n)
    for g in range(G):
        for t in range(m):
            js = np.flatnonzero(see[t])
            if js.size == 0:
                continue
            e = (k[js] @ q[g, t]) * s
            top = e.max()
            p = np.exp(e - top)
            z = p.sum()
            w = p / z
            out[g, t] = w @ v[js]
            mean_abs[g, t] = w @ np.abs(v[js])
            lse[g, t] = top + math.log(z)
            size[g, t] = (np.abs(k[js]) @ np.abs(q[g, t])).max() * s
            weight[js] += w
    return dict(out=out, lse=lse, weight=weight, mean_abs=mean_abs, abs_logit=size)


def evict_segment(pos: np.ndarray, acc: np.ndarray, seen: int, m: int, *, budget: int, n_sink: int, n_recent: int):
    """Rows of the new segment: a list of (old row) for the kept ones, in their new order, before
    the m appended rows."""
    n = len(pos)
    keep = min(n, budget - m)

    def rank(i):
        if pos[i] < n_sink or pos[i] >= seen + m - n_recent:
            return (0, 0.0, i)
        if np.isnan(acc[i]):
            return (2, 0.0, i)
        return (1, -float(acc[i]), i)

    stay = set(sorted(range(n), key=rank)[:keep])
    fills = iter([i for i in range(keep, n) if i in stay])
    return [i if i in stay else next(fills) for i in range(keep)]
