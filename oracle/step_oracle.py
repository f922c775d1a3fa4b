"""64-bit CPU oracle of a step of drafted tokens over the cache: trees and their attention, verification,
pages that requests share, kept rows left in their cache, rotary positions.

TEST INFRASTRUCTURE ONLY (see oracle/kvsel_oracle.py): plain restatements of the definitions, one
request or segment at a time, sharing no code with the CUDA library.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np


# ------------------------------------------------------------------------------ trees
def ancestors(parents) -> np.ndarray:
    """[m][m] bool: node t sees node u (itself and its ancestors); a parent outside [0, t) is none."""
    m = len(parents)
    see = np.eye(m, dtype=bool)
    for t in range(m):
        u = t
        while 0 <= parents[u] < u:
            u = parents[u]
            see[t, u] = True
    return see


def words(see: np.ndarray, n_new: int) -> np.ndarray:
    """Masks as [m][ceil(n_new / 32)] uint32."""
    out = np.zeros((see.shape[0], -(-n_new // 32)), np.uint32)
    for t, u in zip(*np.nonzero(see)):
        out[t, u // 32] |= np.uint32(1 << (u % 32))
    return out


def tree_visible(n: int, see: np.ndarray, window: int, n_sink: int) -> np.ndarray:
    """[m][n]: node t sees cached row j (the tree's rows are the last m of n)."""
    m = see.shape[0]
    out = np.zeros((m, n), bool)
    for t in range(m):
        r = n - m + max(int(see[t].sum()), 1) - 1
        for j in range(n):
            if j >= n - m:
                out[t, j] = see[t, j - (n - m)]
            else:
                out[t, j] = not window or j > r - window or j < n_sink
    return out


def tree_windowed(n: int, see: np.ndarray, window: int, n_sink: int) -> np.ndarray:
    """The same where the window counts the tree's rows too: what a node sees of them lies, in order, at positions
    n - m, n - m + 1, ..."""
    m = see.shape[0]
    out = tree_visible(n, see, window, n_sink)
    for t in range(m):
        line = [int(u) for u in np.flatnonzero(see[t])]
        r = n - m + max(len(line), 1) - 1
        for at, u in enumerate(line, start=n - m):
            if n - m + u >= 0 and window and not (at > r - window or at < n_sink):
                out[t, n - m + u] = False
    return out


def attend_seen(q, k, v, see, scale=None) -> dict:
    """q [G][m][d], k and v [n][d], see [m][n] -> out, lse, and what rounding errors scale with."""
    G, m, d = q.shape
    s = scale or 1.0 / math.sqrt(d)
    out, mean_abs = np.zeros((G, m, d)), np.zeros((G, m, d))
    lse, size = np.full((G, m), -np.inf), np.zeros((G, m))
    for t in range(m):
        js = np.flatnonzero(see[t])
        if js.size == 0:
            continue
        e = (q[:, t] @ k[js].T) * s
        top = e.max(axis=1, keepdims=True)
        p = np.exp(e - top)
        z = p.sum(axis=1, keepdims=True)
        out[:, t], mean_abs[:, t] = (p / z) @ v[js], (p / z) @ np.abs(v[js])
        lse[:, t] = (top + np.log(z))[:, 0]
        size[:, t] = (np.abs(q[:, t]) @ np.abs(k[js]).T).max(axis=1) * s
    return dict(out=out, lse=lse, mean_abs=mean_abs, abs_logit=size)


# ------------------------------------------------------------------------------ verification
def verify(tokens, parents, p, q, u, mode: str):
    """One request: (accepted nodes, next token).  p, q: rows of float values; exact rational arithmetic
    decides (q is None unless sampled)."""
    m, V = len(tokens), len(p[0]) if len(p) else 0
    if m == 0:
        return [], -1
    frac = lambda row: [Fraction(float(x)) for x in row]   # noqa: E731
    c, path = 0, [0]
    while True:
        kids = [t for t in range(1, m) if parents[t] == c]
        taken = None
        if mode == "greedy":
            row = [-math.inf if math.isnan(x) else float(x) for x in p[c]]
            best = row.index(max(row))
            taken = next((t for t in kids if tokens[t] == best), None)
        else:
            r, Z = frac(p[c]), Fraction(1)
            qc = frac(q[c]) if q is not None else None
            for t in kids:
                x = tokens[t]
                if not 0 <= x < V:
                    continue
                if Fraction(float(u[t])) * (qc[x] if qc else 1) * Z < r[x]:
                    taken = t
                    break
                if qc:
                    r = [max(a - Z * b, Fraction(0)) for a, b in zip(r, qc)]
                    Z = sum(r)
                else:
                    Z -= r[x]
                    r[x] = Fraction(0)
        if taken is None:
            break
        c = taken
        path.append(c)
    if mode == "greedy":
        return path, best
    if sum(r) == 0:
        r = frac(p[c])
    goal, at = Fraction(float(u[0])) * sum(r), Fraction(0)
    for x, w in enumerate(r):
        at += w
        if at > goal:
            return path, x
    return path, -1


# ------------------------------------------------------------------------------ pages
class Pages:
    """A block table, the uses of its pages and the pools of every layer, one request after another."""

    def __init__(self, table, ref, k, v):
        self.table, self.ref, self.k, self.v = table.copy(), ref.copy(), k.copy(), v.copy()   # k, v [L][pages][bs][H][d]
        self.bs = k.shape[2]

    def fork(self, src):
        old = self.table.copy()
        for b, s in enumerate(src):
            self.table[b] = old[s] if s >= 0 else -1
            for page in self.table[b][self.table[b] >= 0]:
                self.ref[page] += 1
        for page in old[old >= 0]:
            self.ref[page] -= 1

    def reserve(self, lens, new):
        """lens [B][H] (rows of every head) or [B]."""
        granted, jobs, uses = [], [], self.ref.copy()
        cap = self.table.shape[1] * self.bs
        lens = np.asarray(lens).reshape(len(self.table), -1)
        for b, m in enumerate(new):
            lo, hi = int(lens[b].min()), int(lens[b].max())
            job, keep = [], False
            if hi + m > cap:
                jobs.append(None)
                continue
            if m > 0:
                for i in range(lo // self.bs, -(-(hi + m) // self.bs)):
                    page = self.table[b, i]
                    if page < 0:
                        job.append((i, -1, 0))
                    elif uses[page] > 1:
                        job.append((i, page, min(self.bs, max(0, hi - i * self.bs))))
                        uses[page] -= 1
                    elif self.ref[page] > 1:          # those before it leave it
                        keep = True
            jobs.append((job, keep))
        free, asked = list(np.flatnonzero(self.ref == 0)), 0
        have = len(free)
        for b, x in enumerate(jobs):
            if x is None:
                granted.append(0)
                continue
            job, keep = x
            asked += len(job)
            if (job or keep) and asked > have:
                granted.append(0)
                continue
            for i, page, rows in job:
                to = free.pop(0)
                if page >= 0:
                    for x in (self.k, self.v):
                        x[:, to, :rows] = x[:, page, :rows]
                    self.ref[page] -= 1
                self.table[b, i] = to
                self.ref[to] = 1
            granted.append(int(new[b]))
        return np.array(granted)

    def trim(self, lens):
        lens = np.asarray(lens).reshape(len(self.table), -1)
        for b in range(len(self.table)):
            for i in range(-(-int(lens[b].max()) // self.bs), self.table.shape[1]):
                if self.table[b, i] >= 0:
                    self.ref[self.table[b, i]] -= 1
                    self.table[b, i] = -1

    def accept(self, lens, new, paths):
        """lens [B] or [B][H] with the trees' rows; paths: accepted nodes of every request.  Rows after."""
        out = np.array(lens).copy()
        for b, path in enumerate(paths):
            for h in range(self.k.shape[3]):
                n = int(out[b] if np.ndim(lens) == 1 else lens[b][h])
                base = n - new[b]
                for i, x in enumerate(path):
                    (p0, s0), (p1, s1) = divmod(base + x, self.bs), divmod(base + i, self.bs)
                    for pool in (self.k, self.v):
                        pool[:, self.table[b, p1], s1, h] = pool[:, self.table[b, p0], s0, h]
        for b, path in enumerate(paths):
            out[b] = out[b] - new[b] + len(path)
        return out


def keep_rows(n: int, idx) -> list:
    """Kept positions idx (ascending) of n rows: the position that each of the first len(idx) rows then holds."""
    count = len(idx)
    rows = [i if i in set(idx) else None for i in range(count)]
    fills = [i for i in idx if i >= count]
    return [fills.pop(0) if r is None else r for r in rows]


# ------------------------------------------------------------------------------ rotary positions
def frequencies(rot, theta, scaling="none", factor=1.0, orig_len=0, beta_fast=32.0, beta_slow=1.0, low=1.0, high=4.0):
    """(radians per position of every pair, factor of the values)."""
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = [theta ** (-2 * i / rot) for i in range(rot // 2)]
    scale = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "yarn":
        # the pair whose wave length is orig_len / beta
        pair = lambda beta: rot / 2 * math.log(orig_len / (2 * math.pi * beta)) / math.log(theta)   # noqa: E731
        a, b = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot - 1)
        ramp = [min(max((i - a) / max(b - a, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        f = [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)]
        scale = 0.1 * math.log(factor) + 1
    elif scaling == "bands":
        g = []
        for x in f:
            wave = 2 * math.pi / x
            if wave < orig_len / high:
                g.append(x)
            elif wave > orig_len / low:
                g.append(x / factor)
            else:
                s = (orig_len / wave - low) / (high - low)
                g.append((1 - s) * x / factor + s * x)
        f = g
    return np.array(f), scale


def rope(x, pos, f, scale=1.0, interleaved=False, direction="forward"):
    """x [..., 128], pos [...]: pairs as complex numbers."""
    rot = 2 * len(f)
    a, b = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(rot // 2), np.arange(rot // 2, rot))
    sign = 1.0 if direction == "forward" else -1.0
    grow = 1 / scale if direction == "inverse" else scale
    z = (x[..., a] + 1j * x[..., b]) * (grow * np.exp(1j * sign * np.asarray(pos, np.float64)[..., None] * f))
    y = np.array(x, np.float64)
    y[..., a], y[..., b] = z.real, z.imag
    return y
