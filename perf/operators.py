"""Attention of new tokens over a KV cache, and eviction by accumulated attention weight: the
measured cases, their plain forms in elementary torch operations, and their definitions in
64 bits.

A segment is the cache of one (request, KV head): ``len`` rows of K and V, the last ``m`` of them
the rows of the m new tokens.  Token t (row r = len - m + t) sees row j when j <= r and, with a
window W, j > r - W or j < n_sink.

  attend       out = softmax(q K^T / sqrt(d)) V over the rows that a token sees, and the rows'
               log-sum-exp; with ``acc`` each cached row's weight, summed over tokens and the
               query heads of its group, is added to the row's running total
  evict        makes room for m new rows: keeps the rows with the largest running totals (first
               and recent positions always), moves kept rows from behind into the holes, and
               appends the new rows
"""
import math

import torch

own = False

D = 128
DEV = "cuda"


def listed():
    return [
        # one short chat at the decode step, one layer of the 8-KV-head shape: latency alone counts
        _attend("decode-short", batch=1, h_kv=8, group=4, n_new=1, len_min=1111, len_max=1111),
        # decode step of the ragged serving batch over the paged cache
        _attend("decode-paged-batch", batch=16, h_kv=8, group=4, n_new=1, len_min=2048, len_max=65536, cache="paged", block=16),
        # decode over what a per-layer budget of 10% left of 128K tokens: another length for each head
        _attend("decode-compacted", batch=1, h_kv=4, group=7, n_new=1, len_min=6553, len_max=19661, cache="packed", per_head=True),
        # decode far into a long text that keeps a few first tokens and a window
        _attend("decode-window", batch=8, h_kv=8, group=8, n_new=1, len_min=16384, len_max=65536, cache="paged", block=64, window=4096, n_sink=4),
        # a few drafted tokens checked at once, odd lengths
        _attend("verify-draft", batch=4, h_kv=4, group=7, n_new=6, len_min=3001, len_max=12345, cache="paged", block=32),
        # a 2K chunk of a 32K prompt over the paged cache
        _attend("chunk-paged", batch=1, h_kv=8, group=4, n_new=2048, len_min=32768, len_max=32768, cache="paged", block=16),
        # the last, ragged chunks of four prompts; queries are a slice of the projection's output
        _attend("chunk-ragged", batch=4, h_kv=4, group=7, n_new=517, len_min=2100, len_max=8191, ragged_new=True, token_major=True),
        # a chunk of a long text that keeps a few first tokens and a window
        _attend("chunk-window", batch=1, h_kv=8, group=8, n_new=2048, len_min=16384, len_max=16384, cache="paged", block=16, window=4096, n_sink=4),
        # decode step of a batch whose caches are kept at their budget by accumulated weight
        _attend("accumulate-decode", batch=16, h_kv=8, group=4, n_new=1, len_min=3500, len_max=8192, per_head=True, acc=True),
        # a prefill chunk over such a cache
        _attend("accumulate-chunk", batch=1, h_kv=8, group=4, n_new=1024, len_min=8192, len_max=8192, per_head=True, acc=True),
        # making room for one token in each cache of a batch
        _evict("evict-step", batch=32, h_kv=8, n_new=1, budget=4096, n_sink=4, n_recent=256),
        # making room for a prefill chunk
        _evict("evict-chunk", batch=4, h_kv=8, n_new=2048, budget=16384, n_sink=4, n_recent=2048),
    ]


def _attend(name, *, batch, h_kv, group, n_new, len_min, len_max, cache="contiguous", block=0, window=0, n_sink=0,
            per_head=False, acc=False, ragged_new=False, token_major=False):
    c = dict(op="attend", batch=batch, h_kv=h_kv, group=group, n_new=n_new, len_min=len_min, len_max=len_max, cache=cache,
             block=block, window=window, n_sink=n_sink, per_head=per_head, acc=acc, ragged_new=ragged_new, token_major=token_major)
    return c if name is None else dict(c, name=name)


def _evict(name, *, batch, h_kv, n_new, budget, n_sink, n_recent):
    c = dict(op="evict", batch=batch, h_kv=h_kv, n_new=n_new, budget=budget, n_sink=n_sink, n_recent=n_recent)
    return c if name is None else dict(c, name=name)


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    if rng.random() < 0.25:
        h_kv, budget = rng.choice([1, 2, 4, 8]), log(64, 16384)
        n_new = 1 if rng.random() < 0.5 else log(1, max(1, budget // 4))
        n_recent = rng.randrange(0, budget // 2)
        batch = min(log(1, 32), max(1, 4 * 8 * 16384 // (h_kv * budget)))
        return _evict(None, batch=batch, h_kv=h_kv, n_new=n_new, budget=budget, n_sink=rng.choice([0, 1, 4]), n_recent=n_recent)
    h_kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    cache = rng.choice(["contiguous", "paged", "packed"])
    window = log(16, 8192) if rng.random() < 0.3 else 0
    acc = cache != "packed" and rng.random() < 0.35
    n_new = 1 if rng.random() < 0.5 else log(2, 2048)
    per_head = cache == "packed" or rng.random() < 0.3
    len_max = log(max(n_new, 16), 65536)
    # at most the largest listed cases' pairs of query row and key, and cached rows
    len_max = max(n_new, min(len_max, 2 ** 31 // (h_kv * group * n_new)))
    most = min(2 ** 31 // (h_kv * group * n_new * len_max), 2 ** 23 // (h_kv * len_max))
    batch = max(1, min(log(1, 32), most))
    len_min = max(n_new, int(len_max * rng.uniform(0.1, 1.0)))
    return _attend(None, batch=batch, h_kv=h_kv, group=group, n_new=n_new, len_min=len_min, len_max=len_max, cache=cache,
                   block=rng.choice([8, 16, 32, 64]) if cache == "paged" else 0, window=window,
                   n_sink=rng.choice([0, 1, 4, 64]) if window else 0, per_head=per_head, acc=acc,
                   ragged_new=n_new > 1 and rng.random() < 0.4, token_major=rng.random() < 0.5)


# ------------------------------------------------------------------------------ sizes
def _spread(lo, hi, count, salt):
    """`count` lengths in [lo, hi], scattered the same way for every seed (the largest among them)."""
    got = [lo + (((i + 1) * 2654435761 + salt * 40503) % 2 ** 32) * (hi - lo) // 2 ** 32 for i in range(count)]
    got[(salt * 7) % count] = hi
    return got


def _lens(case):
    """Rows of every segment, [batch][h_kv], and new tokens of every request."""
    B, H, m = case["batch"], case["h_kv"], case["n_new"]
    new = _spread(max(1, m // 3), m, B, 5) if case["ragged_new"] else [m] * B
    if case["per_head"]:
        flat = _spread(case["len_min"], case["len_max"], B * H, 3)
        return [flat[b * H:(b + 1) * H] for b in range(B)], new
    return [[n] * H for n in _spread(case["len_min"], case["len_max"], B, 3)], new


def _visible(n, m, W, sink):
    """(rows that some of the m new tokens sees, pairs of token and row that it sees)."""
    if not W:
        return n, m * n - m * (m - 1) // 2
    lo = max(0, n - m - W + 1)
    rows = n - lo + min(sink, lo)
    pairs = 0
    for r in range(n - m, n):
        first = max(0, r - W + 1)
        pairs += r + 1 - first + min(sink, first)
    return rows, pairs


def work(case):
    B, H, m = case["batch"], case["h_kv"], case["n_new"]
    if case["op"] == "evict":
        n = case["budget"]
        # totals and positions read; the evicted share of the kept range refilled; new rows in
        moved = min(m, n) * (n - m) / n
        return {"bytes": B * H * (8.0 * n + 2 * 512.0 * moved + 2 * 512.0 * m), "flops": 0}
    G = case["group"]
    lens, new = _lens(case)
    rows = pairs = tokens = 0
    for b in range(B):
        for h in range(H):
            r, p = _visible(lens[b][h], new[b], case["window"], case["n_sink"])
            rows, pairs, tokens = rows + r, pairs + p * G, tokens + new[b] * G
    return {"bytes": rows * (512.0 + (8 if case["acc"] else 0)) + tokens * (512.0 + 4), "flops": 4.0 * D * pairs}


# ------------------------------------------------------------------------------ inputs
def _gen(seed, tag):
    return torch.Generator(DEV).manual_seed((int(seed) * 1000003 + tag) % 2 ** 62)


def _normal(shape, seed, tag, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed, tag), device=DEV, dtype=torch.float32) * scale).to(torch.bfloat16)


def _keys(rows, seed, tag):
    """Rows of keys: normal, with log-normal norms (sigma 0.5), as trained caches have them."""
    g = torch.exp(0.5 * torch.randn(rows, generator=_gen(seed, tag + 100), device=DEV))
    return (torch.randn((rows, D), generator=_gen(seed, tag), device=DEV) * g[:, None]).to(torch.bfloat16)


def prepare(case, seed):
    B, H, m = case["batch"], case["h_kv"], case["n_new"]
    st = {"case": case}
    if case["op"] == "evict":
        n = case["budget"]
        st["k"], st["v"] = _keys(B * H * n, seed, 1).view(B, H, n, D), _normal((B, H, n, D), seed, 2)
        # positions: first tokens, a scattered middle, the most recent ones; 4 * budget tokens seen
        seen, recent = 4 * n, min(n, case["n_recent"] + m)
        first = min(case["n_sink"], n - recent)
        mid = n - recent - first
        pos = torch.empty((B, H, n), dtype=torch.int32, device=DEV)
        pos[..., :first] = torch.arange(first, dtype=torch.int32, device=DEV)
        pos[..., n - recent:] = torch.arange(seen - recent, seen, dtype=torch.int32, device=DEV)
        if mid:
            u = torch.rand((B, H, seen - recent - first), generator=_gen(seed, 3), device=DEV)
            pos[..., first:n - recent] = (torch.topk(u, mid, dim=-1).indices + first).to(torch.int32)
        st["pos"] = pos
        st["acc"] = torch.exp(1.5 * torch.randn((B, H, n), generator=_gen(seed, 4), device=DEV))
        st["lens"] = torch.full((B, H), n, dtype=torch.int32, device=DEV)
        st["seen"] = torch.full((B, H), seen, dtype=torch.int32, device=DEV)
        st["k_new"], st["v_new"] = _normal((B, H, m, D), seed, 5), _normal((B, H, m, D), seed, 6)
        return st
    G = case["group"]
    lens, new = _lens(case)
    n_max = case["len_max"]
    if case["token_major"]:  # a slice of the projection's output [batch][token][q heads, k heads, v heads]
        st["q"] = _normal((B, m, (G + 2) * H, D), seed, 7, 1.5)[:, :, :G * H].permute(0, 2, 1, 3)
        st["out"] = torch.zeros((B, m, G * H, D), dtype=torch.bfloat16, device=DEV).permute(0, 2, 1, 3)
    else:
        st["q"] = _normal((B, G * H, m, D), seed, 7, 1.5)
        st["out"] = torch.zeros((B, G * H, m, D), dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.zeros((B, G * H, m), dtype=torch.float32, device=DEV)
    st["lens"] = torch.tensor(lens if case["per_head"] else [r[0] for r in lens], dtype=torch.int32, device=DEV)
    st["new_lens"] = torch.tensor(new, dtype=torch.int32, device=DEV) if case["ragged_new"] else None
    st["offsets"] = None
    if case["cache"] == "paged":
        bs = case["block"]
        blocks = -(-n_max // bs)
        order = torch.randperm(B * blocks, generator=_gen(seed, 8), device=DEV).to(torch.int32)
        st["table"] = order.view(B, blocks)
        st["k"] = _keys(B * blocks * bs * H, seed, 1).view(B * blocks, bs, H, D)
        st["v"] = _normal((B * blocks, bs, H, D), seed, 2)
    elif case["cache"] == "packed":
        flat = [n for r in lens for n in r]
        st["offsets"] = torch.tensor([sum(flat[:i]) for i in range(len(flat))], dtype=torch.int64, device=DEV)
        st["k"], st["v"] = _keys(sum(flat), seed, 1), _normal((sum(flat), D), seed, 2)
    else:
        st["k"], st["v"] = _keys(B * H * n_max, seed, 1).view(B, H, n_max, D), _normal((B, H, n_max, D), seed, 2)
    if case["acc"]:
        st["acc"] = torch.exp(1.5 * torch.randn((B, H, n_max), generator=_gen(seed, 4), device=DEV))
    return st


# ------------------------------------------------------------------------------ one pass
def run(st):
    if st["case"]["op"] == "evict":
        return _own_evict(st) if own else _plain_evict(st)
    return _own_attend(st) if own else _plain_attend(st)


def _gathered(st, x, n_max):
    """The cache rows as [batch][h_kv][n_max][d], 32 bits (rows past a segment's end: any cached row)."""
    case = st["case"]
    B, H = case["batch"], case["h_kv"]
    if case["cache"] == "paged":
        rows = x[st["table"].long()].reshape(B, -1, H, D)[:, :n_max]
        return rows.permute(0, 2, 1, 3).float()
    if case["cache"] == "packed":
        at = st["offsets"].view(B, H, 1) + torch.arange(n_max, device=DEV)
        return x[at.clamp(max=x.shape[0] - 1)].float()
    return x.float()


def _plain_attend(st):
    case = st["case"]
    B, H, G, m = case["batch"], case["h_kv"], case["group"], case["n_new"]
    n_max = case["len_max"]
    lens = st["lens"].view(B, -1, 1, 1, 1).expand(B, H, 1, 1, 1).long()
    new = torch.full((B,), m, device=DEV) if st["new_lens"] is None else st["new_lens"].long()
    t = torch.arange(m, device=DEV).view(1, 1, 1, m, 1)
    j = torch.arange(n_max, device=DEV)
    r = lens - new.view(B, 1, 1, 1, 1) + t
    sees = j <= r
    if case["window"]:
        sees = sees & ((j > r - case["window"]) | (j < case["n_sink"]))
    sees = sees & (t < new.view(B, 1, 1, 1, 1))
    k, v = _gathered(st, st["k"], n_max), _gathered(st, st["v"], n_max)
    q = st["q"].reshape(B, H, G * m, D).float()
    s = torch.matmul(q, k.transpose(2, 3)).view(B, H, G, m, n_max)
    s = s.mul_(1.0 / math.sqrt(D)).masked_fill_(~sees, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    z = p.sum(-1, keepdim=True)
    lse = (top + z.log()).view(B, G * H, m)
    p = p.div_(torch.where(z > 0, z, torch.ones_like(z)))
    o = torch.matmul(p.view(B, H, G * m, n_max), v).view(B, G * H, m, D)
    live = (t.view(1, 1, m) < new.view(B, 1, 1)).expand(B, G * H, m)
    got = {"out": torch.where(live[..., None], o, torch.zeros_like(o)).to(torch.bfloat16),
           "lse": torch.where(live, lse, torch.zeros_like(lse))}
    if case["acc"]:
        st["acc"] += p.sum((2, 3))
        got["acc"] = st["acc"]
    return got


def _plain_evict(st):
    case = st["case"]
    m, budget = case["n_new"], case["budget"]
    pos, acc, k, v = st["pos"], st["acc"], st["k"], st["v"]
    n, seen = st["lens"].long().unsqueeze(-1), st["seen"].unsqueeze(-1)
    keep = torch.minimum(n, torch.full_like(n, budget - m))
    slot = torch.arange(acc.shape[-1], device=DEV).expand_as(acc)
    fixed = (pos < case["n_sink"]) | (pos >= seen + m - case["n_recent"])
    key = torch.where(fixed, torch.full_like(acc, math.inf), acc)
    key = torch.where(slot < n, key, torch.full_like(acc, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(order, dtype=torch.bool).scatter_(-1, order, slot < keep)
    hole = (~kept & (slot < keep)).nonzero(as_tuple=True)
    fill = (kept & (slot >= keep)).nonzero(as_tuple=True)
    pos[hole], acc[hole], k[hole], v[hole] = pos[fill], acc[fill], k[fill], v[fill]
    at = keep + torch.arange(m, device=DEV)
    pos.scatter_(-1, at, seen + torch.arange(m, device=DEV, dtype=torch.int32))
    acc.scatter_(-1, at, 0.0)
    wide = at.unsqueeze(-1).expand(*at.shape, D)
    k.scatter_(2, wide, st["k_new"])
    v.scatter_(2, wide, st["v_new"])
    st["lens"].copy_(keep.squeeze(-1) + m)
    st["seen"] += m
    return {name: st[name] for name in ("k", "v", "pos", "acc", "lens", "seen")}


def _own_attend(st):
    from kv_cache_eviction_window_gb300 import binding

    case = st["case"]
    if "plan" not in st:  # what a program keeps from step to step: parameters, cache view, workspace
        q, out = st["q"], st["out"]
        st["plan"] = binding.make_attn_params(
            h_kv=case["h_kv"], group=case["group"], batch=case["batch"], n_new=case["n_new"], max_len=case["len_max"],
            window=case["window"], n_sink=case["n_sink"], lens_per_head=case["per_head"],
            q_strides=q.stride()[:3], o_strides=out.stride()[:3],
            n_rows=st["k"].shape[0] if case["cache"] == "packed" else 0,
            acc_stride=st["acc"].shape[-1] if case["acc"] else 0)
        if case["cache"] == "paged":
            st["kv"] = binding.make_kv_paged(st["k"], st["v"], st["table"])
        elif case["cache"] == "packed":
            st["kv"] = binding.make_kv_packed(st["k"], st["v"])
        else:
            st["kv"] = binding.make_kv_contiguous(st["k"], st["v"])
        st["ws"] = torch.empty(binding.kvsel_attend_workspace_size(st["plan"], acc=case["acc"]), dtype=torch.uint8, device=DEV)
        binding.kvsel_workspace_init(st["ws"])
    binding.kvsel_attend(st["plan"], st["q"], st["kv"], st["lens"], st["out"], st["ws"], new_lens=st["new_lens"],
                         offsets=st["offsets"], lse=st["lse"], acc=st.get("acc"))
    return {name: st[name] for name in ("out", "lse", "acc") if name in st}


def _own_evict(st):
    from kv_cache_eviction_window_gb300 import binding

    case = st["case"]
    if "plan" not in st:
        st["plan"] = binding.make_evict_params(
            h_kv=case["h_kv"], batch=case["batch"], n_new=case["n_new"], capacity=st["k"].shape[2], budget=case["budget"],
            n_sink=case["n_sink"], n_recent=case["n_recent"])
        st["kv"] = binding.make_kv_contiguous(st["k"], st["v"])
        st["ws"] = torch.empty(binding.kvsel_evict_append_workspace_size(st["plan"]), dtype=torch.uint8, device=DEV)
        binding.kvsel_workspace_init(st["ws"])
    binding.kvsel_evict_append(st["plan"], st["kv"], st["lens"], st["seen"], st["pos"], st["acc"], st["k_new"], st["v_new"],
                               st["ws"])
    return {name: st[name] for name in ("k", "v", "pos", "acc", "lens", "seen")}


# ------------------------------------------------------------------------------ definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return _exact_evict(case, st) if case["op"] == "evict" else _exact_attend(case, st)


def _exact_attend(case, st):
    B, H, G, m = case["batch"], case["h_kv"], case["group"], case["n_new"]
    lens, new = _lens(case)
    out = torch.zeros((B, G * H, m, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, G * H, m), dtype=torch.float64, device=DEV)
    acc = st["acc"].double() if case["acc"] else None
    for b in range(B):
        for h in range(H):
            n, fresh = lens[b][h], new[b]
            if case["cache"] == "paged":
                pages = st["table"][b, :-(-n // case["block"])].long()
                k, v = (st[x][pages, :, h].reshape(-1, D)[:n].double() for x in "kv")
            elif case["cache"] == "packed":
                at = sum(sum(r) for r in lens[:b]) + sum(lens[b][:h])
                k, v = (st[x][at:at + n].double() for x in "kv")
            else:
                k, v = (st[x][b, h, :n].double() for x in "kv")
            row = torch.arange(n - fresh, n, device=DEV)[:, None]
            col = torch.arange(n, device=DEV)[None, :]
            hidden = col > row
            if case["window"]:
                hidden |= (row - col >= case["window"]) & (col >= case["n_sink"])
            for g in range(G):
                e = st["q"][b, h * G + g, :fresh].double() @ k.T / math.sqrt(D)
                e[hidden] = -math.inf
                norm = torch.logsumexp(e, 1)
                w = torch.exp(e - norm[:, None])
                out[b, h * G + g, :fresh] = w @ v
                lse[b, h * G + g, :fresh] = norm
                if acc is not None:
                    acc[b, h, :n] += w.sum(0)
    return {"out": out, "lse": lse} | ({} if acc is None else {"acc": acc})


def _exact_evict(case, st):
    B, H, m, budget = case["batch"], case["h_kv"], case["n_new"], case["budget"]
    got = {x: st[x].clone() for x in ("k", "v", "pos", "acc", "lens", "seen")}
    for b in range(B):
        for h in range(H):
            n, seen = int(st["lens"][b, h]), int(st["seen"][b, h])
            keep = min(n, budget - m)
            pos, acc = st["pos"][b, h, :n].tolist(), st["acc"][b, h, :n].tolist()

            def rank(i):
                fixed = pos[i] < case["n_sink"] or pos[i] >= seen + m - case["n_recent"]
                return (0, 0.0, i) if fixed else (1, -acc[i], i)

            stay = set(sorted(range(n), key=rank)[:keep])
            holes = [i for i in range(keep) if i not in stay]
            fills = [i for i in range(keep, n) if i in stay]
            if holes:
                to, of = torch.tensor(holes, device=DEV), torch.tensor(fills, device=DEV)
                for x in ("k", "v", "pos", "acc"):
                    got[x][b, h, to] = st[x][b, h, of]
            got["k"][b, h, keep:keep + m] = st["k_new"][b, h]
            got["v"][b, h, keep:keep + m] = st["v_new"][b, h]
            got["pos"][b, h, keep:keep + m] = torch.arange(seen, seen + m, dtype=torch.int32, device=DEV)
            got["acc"][b, h, keep:keep + m] = 0.0
            got["lens"][b, h] = keep + m
            got["seen"][b, h] = seen + m
    return {x: y.double() if y.is_floating_point() else y for x, y in got.items()}
