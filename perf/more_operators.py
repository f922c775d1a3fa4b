"""A step of drafted tokens over the cache: attention of a tree, verification, accepted rows and the
pages that requests share, rotary positions.  The measured cases, their plain forms in elementary
torch operations, and their definitions in 64 bits.

A tree has m nodes per request: node 0 the token decided last, the others drafted, parents before
children.  Its rows are the last m of a segment (the cache of one request and KV head, n rows).

  tree      out = softmax(q K^T / sqrt(d)) V: node t sees the rows before the tree (with a window W
            those of the last W positions and the first n_sink) and row u of the tree where bit u of
            its mask is set (itself and its ancestors); its position is n - m + set bits - 1
  verify    walks from node 0: a child is accepted with probability min(1, r(x) / (Z q(x))), each
            rejection takes q from the rest r = max(r - Z q, 0), and the token after the last
            accepted node is drawn from r (point: q is 1 at the drafted token; greedy: the child that
            has the target's largest value is accepted)
  beam      table rows are taken from other rows, pages are counted by their uses, and rows for new
            tokens are reserved: a last page that others use too is copied
  accept    rows of new tokens are reserved, the accepted rows of the tree move to its front in every
            layer, and the pages behind them are free again
  keep      a selection's rows stay in their cache: those behind the kept number fill the holes
  rope      rows are rotated by their positions (frequencies scaled for long contexts)
  unrope    cached keys as they were before their rotation
"""
import math
import random

import torch

own = False

D = 128
DEV = "cuda"


def listed():
    return [
        # one short chat: 16 drafted tokens of one request, the step's first layer (with the masks of the tree)
        _tree("tree-short", batch=1, h_kv=8, group=4, nodes=16, len_min=1111, len_max=1111, cache="contiguous", masks=True),
        # a ragged serving batch over the paged cache, 32 drafted tokens each
        _tree("tree-batch", batch=8, h_kv=8, group=4, nodes=32, len_min=2048, len_max=32768, block=16),
        # a wide tree far into one long text
        _tree("tree-long", batch=1, h_kv=8, group=4, nodes=64, len_min=131072, len_max=131072, block=64),
        # ragged trees of a model whose layers see a window and a few first tokens, odd group and lengths
        _tree("tree-window", batch=5, h_kv=4, group=7, nodes=26, len_min=3001, len_max=24001, block=32, window=4096, n_sink=4, ragged=True),
        # five drafted tokens of each request of a batch, a chain
        _verify("verify-chain", batch=32, nodes=6, vocab=50257, mode="sampled", shape="chain"),
        # trees whose siblings were drawn independently, the large vocabulary, bf16 probabilities
        _verify("verify-tree", batch=8, nodes=64, vocab=131072, mode="sampled", dtype="bf16"),
        # greedy decoding of a batch by its logits
        _verify("verify-greedy", batch=32, nodes=26, vocab=131072, mode="greedy", dtype="bf16", ragged=True),
        # 16 prompts of four beams: one step of the search
        _pages("beam-step", "beam", batch=64, width=4, h_kv=8, layers=8, len_min=500, len_max=2000, block=16, n_new=1),
        # the step after a verification, every layer's pool
        _pages("accept-step", "accept", batch=32, width=1, h_kv=8, layers=8, len_min=300, len_max=1300, block=16, n_new=32),
        # 40% of 32K tokens stay after the prompt, another set for each head, in place
        _keep("keep-32k", batch=4, h_kv=8, n=32768, ratio=0.4, block=16),
        # queries and keys of a prompt's chunk, slices of the projection's output, far positions
        _rope("rope-chunk", batch=2, h_q=32, h_kv=8, n_new=4096, scaling="yarn", factor=16.0, first=131072),
        # pre-rotation keys of an evicted cache's rows
        _unrope("unrope-cache", batch=4, h_kv=8, n=13107, block=16, scaling="bands", factor=8.0, interleaved=False, rot=128),
    ]


def _named(name, c):
    return c if name is None else dict(c, name=name)


def _tree(name, *, batch, h_kv, group, nodes, len_min, len_max, cache="paged", block=0, window=0, n_sink=0, ragged=False, masks=False):
    return _named(name, dict(op="tree", batch=batch, h_kv=h_kv, group=group, nodes=nodes, len_min=len_min, len_max=len_max, cache=cache,
                             block=block, window=window, n_sink=n_sink, ragged=ragged, masks=masks))


def _verify(name, *, batch, nodes, vocab, mode, dtype="fp32", shape="tree", ragged=False):
    return _named(name, dict(op="verify", batch=batch, nodes=nodes, vocab=vocab, mode=mode, dtype=dtype, shape=shape, ragged=ragged))


def _pages(name, op, *, batch, width, h_kv, layers, len_min, len_max, block, n_new):
    return _named(name, dict(op=op, batch=batch, width=width, h_kv=h_kv, layers=layers, len_min=len_min, len_max=len_max, block=block, n_new=n_new))


def _keep(name, *, batch, h_kv, n, ratio, block):
    return _named(name, dict(op="keep", batch=batch, h_kv=h_kv, n=n, ratio=ratio, block=block))


def _rope(name, *, batch, h_q, h_kv, n_new, scaling="none", factor=1.0, first=0, interleaved=False, rot=128, direction="forward"):
    return _named(name, dict(op="rope", batch=batch, h_q=h_q, h_kv=h_kv, n_new=n_new, scaling=scaling, factor=factor, first=first,
                             interleaved=interleaved, rot=rot, direction=direction))


def _unrope(name, *, batch, h_kv, n, block, scaling, factor, interleaved, rot):
    return _named(name, dict(op="unrope", batch=batch, h_kv=h_kv, n=n, block=block, scaling=scaling, factor=factor, interleaved=interleaved, rot=rot))


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["tree", "tree", "tree", "verify", "verify", "beam", "accept", "keep", "rope", "unrope"])
    if kind == "tree":
        h_kv, group, nodes = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16]), log(1, 128)
        window = log(16, 8192) if rng.random() < 0.3 else 0
        cache = rng.choice(["contiguous", "paged", "paged"])
        # at most the largest listed cases' pairs of query row and key, and cached rows
        len_max = max(nodes, min(log(max(nodes, 16), 131072), 2 ** 28 // (h_kv * group * nodes)))
        most = min(2 ** 28 // (h_kv * group * nodes * len_max), 2 ** 20 // (h_kv * len_max))
        return _tree(None, batch=max(1, min(log(1, 32), most)), h_kv=h_kv, group=group, nodes=nodes, len_min=max(nodes, int(len_max * rng.uniform(0.1, 1.0))),
                     len_max=len_max, cache=cache, block=rng.choice([8, 16, 32, 64]) if cache == "paged" else 0, window=window,
                     n_sink=rng.choice([0, 1, 4, 64]) if window else 0, ragged=rng.random() < 0.4, masks=rng.random() < 0.2)
    if kind == "verify":
        vocab, nodes = log(1000, 131072), log(1, 64)
        return _verify(None, batch=max(1, min(log(1, 64), 2 ** 26 // (vocab * nodes))), nodes=nodes, vocab=vocab, mode=rng.choice(["sampled", "sampled", "point", "greedy"]),
                       dtype=rng.choice(["fp32", "bf16"]), shape=rng.choice(["chain", "tree"]), ragged=rng.random() < 0.4)
    if kind in ("beam", "accept"):
        h_kv, layers, block = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8]), rng.choice([8, 16, 32, 64])
        width = rng.choice([1, 2, 4, 5]) if kind == "beam" else 1
        len_max = log(20, 2000)
        prompts = max(1, min(log(1, 32), 2 ** 18 // (len_max * h_kv * layers)))
        return _pages(None, kind, batch=prompts * width, width=width, h_kv=h_kv, layers=layers, len_min=max(1, int(len_max * rng.uniform(0.1, 1.0))), len_max=len_max,
                      block=block, n_new=1 if kind == "beam" else log(2, 64))
    if kind == "keep":
        h_kv, n = rng.choice([1, 2, 4, 8]), log(64, 32768)
        return _keep(None, batch=max(1, min(log(1, 16), 2 ** 20 // (h_kv * n))), h_kv=h_kv, n=n, ratio=rng.uniform(0.05, 0.95), block=rng.choice([0, 8, 16, 32, 64]))
    scaling = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
    factor = 1.0 if scaling == "none" else rng.uniform(1.5, 32.0)
    rot, interleaved = rng.choice([32, 64, 96, 128, 128, 128]), rng.random() < 0.5
    if kind == "rope":
        h_kv, n_new = rng.choice([1, 2, 4, 8]), log(1, 4096)
        h_q = h_kv * rng.choice([1, 2, 4, 7])
        return _rope(None, batch=max(1, min(log(1, 64), 2 ** 18 // (n_new * (h_q + h_kv)))), h_q=h_q, h_kv=h_kv, n_new=n_new, scaling=scaling, factor=factor,
                     first=log(1, 2 ** 20), interleaved=interleaved, rot=rot, direction=rng.choice(["forward", "transpose", "inverse"]))
    h_kv, n = rng.choice([1, 2, 4, 8]), log(64, 32768)
    return _unrope(None, batch=max(1, min(log(1, 16), 2 ** 18 // (h_kv * n))), h_kv=h_kv, n=n, block=rng.choice([0, 8, 16, 32, 64]), scaling=scaling, factor=factor,
                   interleaved=interleaved, rot=rot)


# ------------------------------------------------------------------------------ sizes
def _spread(lo, hi, count, salt):
    """`count` lengths in [lo, hi], scattered the same way for every seed (the largest among them)."""
    got = [lo + (((i + 1) * 2654435761 + salt * 40503) % 2 ** 32) * (hi - lo) // 2 ** 32 for i in range(count)]
    got[(salt * 7) % count] = hi
    return got


def _sizes(case):
    """Rows of every request, and nodes of its tree."""
    B, m = case["batch"], case["nodes"]
    return _spread(case["len_min"], case["len_max"], B, 3) if "len_min" in case else None, _spread(max(1, m // 3), m, B, 5) if case["ragged"] else [m] * B


def _prompts(case):
    """Rows of the requests of a page case, the same for the beams of a prompt."""
    w = case["width"]
    return [n for n in _spread(case["len_min"], case["len_max"], case["batch"] // w, 3) for _ in range(w)]


def _cap(case):
    """Pages of a request at most."""
    return -(-(case["len_max"] + case["n_new"]) // case["block"]) + 1


def work(case):
    op = case["op"]
    if op == "tree":
        lens, new = _sizes(case)
        rows = pairs = 0
        for n, m in zip(lens, new):
            seen = n - m if not case["window"] else min(n - m, case["window"] + case["n_sink"])
            rows += seen + m
            pairs += (seen + 1) * m
        H, G = case["h_kv"], case["group"]
        return {"bytes": H * (512.0 * rows + G * sum(new) * 516.0), "flops": 4.0 * D * H * G * pairs}
    if op == "verify":
        # at least one row of the target's values (and of the draft's) is read whole for every request
        size = 4.0 if case["dtype"] == "fp32" else 2.0
        return {"bytes": case["batch"] * (case["vocab"] * size * (2 if case["mode"] == "sampled" else 1) + 12.0 * case["nodes"]), "flops": 0}
    if op in ("beam", "accept"):
        row = case["layers"] * case["h_kv"] * 512.0
        lens = _prompts(case)
        if op == "beam":      # a beam in four, about, keeps its last page to itself
            moved = sum(n % case["block"] for n in lens) * (1 - 1 / case["width"])
            tables = 2 * 4.0 * sum(-(-n // case["block"]) for n in lens)
        else:                 # two rows of a request move, about
            moved, tables = 2 * len(lens), 3 * 4.0 * len(lens) * -(-case["n_new"] // case["block"])
        return {"bytes": 2 * row * moved + tables, "flops": 0}
    if op == "keep":
        keep = _kept(case)
        moved = keep * (1 - keep / case["n"])
        return {"bytes": case["batch"] * case["h_kv"] * (1024.0 * moved + 12.0 * keep), "flops": 0}
    if op == "rope":
        rows = case["batch"] * case["n_new"] * (case["h_q"] + case["h_kv"])
        return {"bytes": 512.0 * rows + 4.0 * case["batch"] * case["n_new"], "flops": 3.0 * case["rot"] * rows}
    rows = case["batch"] * case["h_kv"] * case["n"]
    return {"bytes": 516.0 * rows, "flops": 3.0 * case["rot"] * rows}


def _kept(case):
    return max(1, int(case["n"] * case["ratio"]))


# ------------------------------------------------------------------------------ inputs
def _gen(seed, tag):
    return torch.Generator(DEV).manual_seed((int(seed) * 1000003 + tag) % 2 ** 62)


def _normal(shape, seed, tag, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed, tag), device=DEV, dtype=torch.float32) * scale).to(torch.bfloat16)


def _keys(rows, seed, tag):
    """Rows of keys: normal, with log-normal norms (sigma 0.5), as trained caches have them."""
    g = torch.exp(0.5 * torch.randn(rows, generator=_gen(seed, tag + 100), device=DEV))
    return (torch.randn((rows, D), generator=_gen(seed, tag), device=DEV) * g[:, None]).to(torch.bfloat16)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _parents(case, seed, new):
    """Parents of the trees' nodes, [batch][nodes]; -1 for node 0 and behind a tree."""
    rng = random.Random(int(seed) * 7919 + 17)
    got = []
    for m in new:
        if case.get("shape") == "chain":
            p = [t - 1 for t in range(m)]
        else:
            p = [-1] + [t - 1 if rng.random() < 0.45 else rng.randrange(t) for t in range(1, m)]
        got.append(p + [-1] * (case["nodes"] - m))
    return got


def _words(parents, nodes):
    """Masks of the trees: [batch][nodes][words], bit u: node u is seen."""
    words = -(-nodes // 32)
    got = []
    for row in parents:
        masks = []
        for t, p in enumerate(row):
            masks.append((masks[p] if p >= 0 else 0) | 1 << t)
        got.append([[(x >> 32 * w & 0xFFFFFFFF) - (2 ** 32 if x >> 32 * w & 0x80000000 else 0) for w in range(words)] for x in masks])
    return _ints(got)


def prepare(case, seed):
    return {"tree": _prepare_tree, "verify": _prepare_verify, "beam": _prepare_pages, "accept": _prepare_pages, "keep": _prepare_keep,
            "rope": _prepare_rope, "unrope": _prepare_unrope}[case["op"]](case, seed, {"case": case})


def _prepare_tree(case, seed, st):
    B, H, G, m, n_max = case["batch"], case["h_kv"], case["group"], case["nodes"], case["len_max"]
    lens, new = _sizes(case)
    st["q"] = _normal((B, G * H, m, D), seed, 7, 1.5)
    st["out"] = torch.zeros((B, G * H, m, D), dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.zeros((B, G * H, m), dtype=torch.float32, device=DEV)
    st["lens"], st["new_lens"] = _ints(lens), _ints(new)
    parents = _parents(case, seed, new)
    st["parents"], st["tree"] = _ints(parents), _words(parents, m)
    st["first"] = _ints([n - k for n, k in zip(lens, new)])
    st["pos"] = torch.zeros((B, m), dtype=torch.int32, device=DEV)
    if case["cache"] == "paged":
        bs = case["block"]
        blocks = -(-n_max // bs)
        st["table"] = torch.randperm(B * blocks, generator=_gen(seed, 8), device=DEV).to(torch.int32).view(B, blocks)
        st["k"] = _keys(B * blocks * bs * H, seed, 1).view(B * blocks, bs, H, D)
        st["v"] = _normal((B * blocks, bs, H, D), seed, 2)
    else:
        st["k"], st["v"] = _keys(B * H * n_max, seed, 1).view(B, H, n_max, D), _normal((B, H, n_max, D), seed, 2)
    return st


def _prepare_verify(case, seed, st):
    B, m, V = case["batch"], case["nodes"], case["vocab"]
    new = _sizes(case)[1]
    kind = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    parents = _parents(case, seed, new)
    st["parents"], st["new_lens"] = _ints(parents), _ints(new)
    at = st["parents"].long().clamp(min=0)
    batch = torch.arange(B, device=DEV)[:, None]
    logits = 2.5 * torch.randn((B, m, V), generator=_gen(seed, 1), device=DEV)
    guess = logits + 0.7 * torch.randn((B, m, V), generator=_gen(seed, 2), device=DEV)
    st["u"] = torch.rand((B, m), generator=_gen(seed, 3), device=DEV)
    st["draft"] = None
    if case["mode"] == "sampled":
        st["target"], st["draft"] = torch.softmax(logits, -1).to(kind), torch.softmax(guess, -1).to(kind)
        pick = torch.rand((B, m), generator=_gen(seed, 4), device=DEV)
        st["tokens"] = torch.zeros((B, m), dtype=torch.int32, device=DEV)
        for t in range(m):    # each child is drawn from its parent's distribution
            c = st["draft"][batch[:, 0], at[:, t]].double().cumsum(-1)
            st["tokens"][:, t] = (c <= (pick[:, t, None].double() * c[:, -1:])).sum(-1).clamp(max=V - 1).to(torch.int32)
    else:                     # a node's children are the draft's likeliest tokens, in order
        rank = [[sum(p == row[t] for p in row[:t]) if t else 0 for t, _ in enumerate(row)] for row in parents]
        best = guess.topk(min(V, max(max(r) for r in rank) + 1), -1).indices
        st["tokens"] = best[batch, at, torch.tensor(rank, device=DEV).clamp(max=best.shape[-1] - 1)].to(torch.int32)
        st["target"] = (logits if case["mode"] == "greedy" else torch.softmax(logits, -1)).to(kind)
    st["path"] = torch.zeros((B, m), dtype=torch.int32, device=DEV)
    st["counts"], st["next"] = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    return st


def _prepare_pages(case, seed, st):
    """Tables in which the beams of a prompt share all pages but the last, pools with free pages in between."""
    B, w, bs, cap = case["batch"], case["width"], case["block"], _cap(case)
    lens = _prompts(case)
    rng = random.Random(int(seed) * 7919 + 23)
    spare = B * (-(-case["n_new"] // bs) + 2)
    total = sum(-(-n // bs) + w - 1 for n in lens[::w]) + spare
    ids = list(range(total))
    rng.shuffle(ids)
    table, ref = [[-1] * cap for _ in range(B)], [0] * total
    for b, n in enumerate(lens):
        used = -(-n // bs)
        for i in range(used):
            shared = b % w and i < used - 1
            table[b][i] = table[b - b % w][i] if shared else ids.pop()
            ref[table[b][i]] += 1
    st["table"] = [_ints(table), _ints([[-1] * cap for _ in range(B)])]
    st["ref"], st["lens"], st["now"] = _ints(ref), [_ints(lens), _ints(lens)], 0
    st["granted"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    shape = (case["layers"], total, bs, case["h_kv"], D)
    st["k"], st["v"] = _normal(shape, seed, 1), _normal(shape, seed, 2)
    if case["op"] == "beam":
        st["src"] = _ints([b - b % w + rng.randrange(w) for b in range(B)])
    else:
        m = case["n_new"]
        st["all"] = _ints([n + m for n in lens])
        path = []
        for _ in range(B):    # a walk down a tree: node 0, then a child with probability 0.7 each time
            p = [0]
            while rng.random() < 0.7 and p[-1] + 1 < m:
                p.append(rng.randrange(p[-1] + 1, min(m, p[-1] + 9)))
            path.append(p)
        st["counts"], st["path"] = _ints([len(p) for p in path]), _ints([p + [-1] * (m - len(p)) for p in path])
    return st


def _prepare_keep(case, seed, st):
    B, H, n, bs, keep = case["batch"], case["h_kv"], case["n"], case["block"], _kept(case)
    if bs:
        blocks = -(-n // bs)
        st["table"] = torch.randperm(B * blocks, generator=_gen(seed, 8), device=DEV).to(torch.int32).view(B, blocks)
        shape = (B * blocks, bs, H, D)
    else:
        shape = (B, H, n, D)
    st["k"], st["v"] = _normal(shape, seed, 1), _normal(shape, seed, 2)
    st["scores"] = torch.exp(1.5 * torch.randn((B, H, n), generator=_gen(seed, 4), device=DEV))
    st["idx"] = st["scores"].topk(keep, -1).indices.sort(-1).values.to(torch.int32).contiguous()
    st["counts"] = torch.full((B, H), keep, dtype=torch.int32, device=DEV)
    st["offsets"] = torch.arange(B * H, device=DEV) * keep
    st["lens"], st["seen"] = torch.zeros((B, H), dtype=torch.int32, device=DEV), torch.zeros((B, H), dtype=torch.int32, device=DEV)
    st["pos"], st["acc"] = torch.zeros((B, H, n), dtype=torch.int32, device=DEV), torch.zeros((B, H, n), device=DEV)
    return st


def _prepare_rope(case, seed, st):
    B, m, hq, hk = case["batch"], case["n_new"], case["h_q"], case["h_kv"]
    st["x"] = _normal((B, m, hq + 2 * hk, D), seed, 1)      # the projection's output: query, key and value heads
    first = torch.randint(case["first"] // 2, case["first"] + 1, (B, 1), generator=_gen(seed, 2), device=DEV)
    st["pos"] = (first + torch.arange(m, device=DEV)).to(torch.int32)
    st["q"], st["k"] = (torch.zeros((B, h, m, D), dtype=torch.bfloat16, device=DEV) for h in (hq, hk))
    return st


def _prepare_unrope(case, seed, st):
    B, H, n, bs = case["batch"], case["h_kv"], case["n"], case["block"]
    if bs:
        blocks = -(-n // bs)
        st["table"] = torch.randperm(B * blocks, generator=_gen(seed, 8), device=DEV).to(torch.int32).view(B, blocks)
        st["key"] = _keys(B * blocks * bs * H, seed, 1).view(B * blocks, bs, H, D)
    else:
        st["key"] = _keys(B * H * n, seed, 1).view(B, H, n, D)
    st["pos"] = torch.randint(0, 4 * n, (B, H, n), generator=_gen(seed, 2), device=DEV, dtype=torch.int32)
    st["lens"] = torch.full((B, H), n, dtype=torch.int32, device=DEV)
    st["out"] = torch.zeros((B, H, n, D), dtype=torch.bfloat16, device=DEV)
    return st


# ------------------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return {"tree": _own_tree, "verify": _own_verify, "beam": _own_beam, "accept": _own_accept, "keep": _own_keep, "rope": _own_rope,
                "unrope": _own_unrope}[op](st)
    return {"tree": _plain_tree, "verify": _plain_verify, "beam": _plain_beam, "accept": _plain_accept, "keep": _plain_keep, "rope": _plain_rope,
            "unrope": _plain_unrope}[op](st)


def _plain_masks(st):
    """Which nodes a node sees, from the parents, and its position."""
    m, par, new = st["case"]["nodes"], st["parents"].long(), st["new_lens"].long()
    own_bit = torch.eye(m, dtype=torch.bool, device=DEV)
    sees, rows = [], torch.arange(len(par), device=DEV)
    for t in range(m):
        up = torch.stack(sees, 1)[rows, par[:, t].clamp(min=0)] if t else torch.zeros_like(own_bit[:1]).expand(len(par), m)
        sees.append((up & (par[:, t] >= 0)[:, None]) | own_bit[t])
    sees = torch.stack(sees, 1)
    bits = sees.long()
    pad = torch.nn.functional.pad(bits, (0, -m % 32)).view(*bits.shape[:2], -1, 32)
    words = (pad << torch.arange(32, device=DEV)).sum(-1)
    live = torch.arange(m, device=DEV) < new[:, None]
    pos = torch.where(live, st["first"][:, None].long() + bits.sum(-1) - 1, st["pos"].long())
    return sees, torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32), pos.to(torch.int32)


def _plain_tree(st):
    case = st["case"]
    B, H, G, m, n_max = case["batch"], case["h_kv"], case["group"], case["nodes"], case["len_max"]
    got = {}
    if case["masks"]:
        sees, words, st["pos"] = _plain_masks(st)
        live = torch.arange(m, device=DEV) < st["new_lens"][:, None]
        got["tree"], got["pos"] = torch.where(live[..., None], words, st["tree"]), st["pos"]
    else:
        u = torch.arange(m, device=DEV)
        sees = (st["tree"].long()[:, :, u // 32] >> (u % 32)) & 1 > 0
    n, new = st["lens"].long().view(B, 1, 1), st["new_lens"].long().view(B, 1, 1)
    t, j = torch.arange(m, device=DEV).view(1, m, 1), torch.arange(n_max, device=DEV)
    sees = sees & (torch.arange(m, device=DEV) < new)
    u = j - (n - new)
    seen = sees.gather(2, u.clamp(0, m - 1).expand(B, m, n_max)) & (u >= 0) & (j < n)
    old = (u < 0).expand(B, m, n_max)
    if case["window"]:
        at = n - new + sees.sum(-1, keepdim=True) - 1
        old = old & ((j > at - case["window"]) | (j < case["n_sink"]))
    seen = ((seen | old) & (t < new)).view(B, 1, 1, m, n_max)
    if case["cache"] == "paged":
        k, v = (st[x][st["table"].long()].reshape(B, -1, H, D)[:, :n_max].permute(0, 2, 1, 3).float() for x in "kv")
    else:
        k, v = st["k"].float(), st["v"].float()
    s = torch.matmul(st["q"].reshape(B, H, G * m, D).float(), k.transpose(2, 3)).view(B, H, G, m, n_max)
    s = s.mul_(1.0 / math.sqrt(D)).masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    z = p.sum(-1, keepdim=True)
    lse = (top + z.log()).view(B, G * H, m)
    p = p.div_(torch.where(z > 0, z, torch.ones_like(z)))
    o = torch.matmul(p.view(B, H, G * m, n_max), v).view(B, G * H, m, D)
    live = (t.view(1, 1, m) < new).expand(B, G * H, m)
    got["out"] = torch.where(live[..., None], o, torch.zeros_like(o)).to(torch.bfloat16)
    got["lse"] = torch.where(live, lse, torch.zeros_like(lse))
    return got


def _plain_verify(st):
    case = st["case"]
    B, m, V = case["batch"], case["nodes"], case["vocab"]
    par, tok, new, mode = st["parents"].long(), st["tokens"].long(), st["new_lens"].long(), case["mode"]
    rows, word = torch.arange(B, device=DEV), torch.arange(V, device=DEV)
    cur = torch.zeros(B, dtype=torch.long, device=DEV)
    count = torch.ones_like(cur)
    path = torch.full((B, m), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    u = st["u"].double()

    def largest(x):
        x = x.float()
        return torch.where(x == x.amax(-1, keepdim=True), word, V).amin(-1)

    rest = st["target"][rows, cur].double()
    mass = torch.ones(B, dtype=torch.float64, device=DEV)
    best = largest(rest) if mode == "greedy" else None
    for t in range(1, m):
        here = (par[:, t] == cur) & (t < new)
        x = tok[:, t]
        if mode == "greedy":
            take = here & (x == best)
        else:
            q = st["draft"][rows, cur].double() if mode == "sampled" else (word == x[:, None]).double()
            px, qx = rest.gather(1, x[:, None])[:, 0], q.gather(1, x[:, None])[:, 0]
            take = here & (u[:, t] * qx * mass < px)
        drop = here & ~take
        cur = torch.where(take, torch.full_like(cur, t), cur)
        path.scatter_(1, torch.where(take, count, torch.zeros_like(count))[:, None], torch.where(take, cur, torch.zeros_like(cur)).to(torch.int32)[:, None])
        count = count + take.long()
        fresh = st["target"][rows, cur].double()
        if mode == "greedy":
            best = largest(fresh)
            continue
        if mode == "sampled":
            less = (rest - mass[:, None] * q).clamp(min=0)
            left = less.sum(-1)
        else:
            less = torch.where(word == x[:, None], torch.zeros_like(rest), rest)
            left = mass - px
        rest = torch.where(take[:, None], fresh, torch.where(drop[:, None], less, rest))
        mass = torch.where(take, torch.ones_like(mass), torch.where(drop, left, mass))
    if mode == "greedy":
        nxt = best
    else:
        c = rest.cumsum(-1)
        c = torch.where(c[:, -1:] > 0, c, st["target"][rows, cur].double().cumsum(-1))
        nxt = (c <= u[:, :1] * c[:, -1:]).sum(-1).clamp(max=V - 1)
    return {"path": path, "counts": count.to(torch.int32), "next": nxt.to(torch.int32)}


def _plain_reserve(st, table, lens):
    """Pages for n_new more rows of every request, the lowest free ones; a page that new rows go to and that
    an earlier request does not leave to this one alone is copied."""
    case = st["case"]
    B, bs, ref = case["batch"], case["block"], st["ref"]
    per = -(-case["n_new"] // bs) + 1
    i = lens.long()[:, None] // bs + torch.arange(per, device=DEV)
    inside = i * bs < lens.long()[:, None] + case["n_new"]
    old = torch.where(inside, table.gather(1, i.clamp(max=table.shape[1] - 1)).long(), -1)
    alike = (old[:, None, :] == old[None, :, :]) & (old >= 0)[None]
    rank = (alike & (torch.arange(B, device=DEV)[:, None] > torch.arange(B, device=DEV))[..., None]).sum(1)
    copied = (old >= 0) & (ref.long()[old.clamp(min=0)] - rank > 1)
    need = inside & ((old < 0) | copied)
    free = torch.sort((ref > 0).to(torch.int32), stable=True).indices
    upto = need.sum(1).cumsum(0)
    served = (upto <= (ref == 0).sum()) | (need.sum(1) == 0)
    need, copied = need & served[:, None], copied & served[:, None]
    order = (need.flatten().long().cumsum(0) - 1).clamp(min=0).view(B, per)
    page = torch.where(need, free[order.clamp(max=len(free) - 1)], old.clamp(min=0))
    # (where nothing is copied, the request's first page is written with what it holds)
    first = table[:, :1].long()
    to, of = torch.where(copied, page, first).flatten(), torch.where(copied, old, first).flatten()
    keep = torch.arange(bs, device=DEV) < torch.where(copied, lens.long()[:, None] - i * bs, 0).clamp(0, bs).flatten()[:, None]
    for x in (st["k"], st["v"]):
        x[:, to] = torch.where(keep[None, :, :, None, None], x[:, of], x[:, to])
    add = torch.zeros_like(ref).scatter_add_(0, page.flatten(), need.flatten().to(torch.int32))
    ref += add.scatter_add_(0, of, -copied.flatten().to(torch.int32))
    wide = torch.cat([table.long(), table.new_zeros((B, 1)).long()], 1)
    wide.scatter_(1, torch.where(need, i, table.shape[1]), page)
    table.copy_(wide[:, :-1])
    st["granted"].copy_(torch.where(served, case["n_new"], 0))


def _plain_beam(st):
    a = st["now"]
    st["now"] = 1 - a
    old, table, src, ref = st["table"][a], st["table"][1 - a], st["src"].long(), st["ref"]
    table.copy_(old[src])
    st["lens"][1 - a].copy_(st["lens"][a][src])
    for x, by in ((table, 1), (old, -1)):
        x = x.flatten().long()
        ref.scatter_add_(0, x.clamp(min=0), torch.where(x >= 0, by, 0).to(torch.int32))
    _plain_reserve(st, table, st["lens"][1 - a])
    return {"table": table, "lens": st["lens"][1 - a], "ref": ref, "granted": st["granted"], "k": st["k"], "v": st["v"]}


def _plain_accept(st):
    case = st["case"]
    B, bs, m, table, ref = case["batch"], case["block"], case["n_new"], st["table"][0], st["ref"]
    _plain_reserve(st, table, st["lens"][0])
    base = (st["all"] - m).long()[:, None]
    i = torch.arange(m, device=DEV)
    live = (i < st["counts"][:, None]) & (st["path"] >= 0)
    of, to = base + torch.where(live, st["path"].long(), i), base + i
    page = [table.gather(1, x // bs).long().clamp(min=0) * bs + x % bs for x in (of, to)]
    for x in (st["k"], st["v"]):
        flat = x.view(case["layers"], -1, case["h_kv"], D)
        flat[:, page[1]] = torch.where(live[None, :, :, None, None], flat[:, page[0]], flat[:, page[1]])
    st["lens"][1].copy_((base[:, 0] + st["counts"]).to(torch.int32))
    pages = torch.arange(table.shape[1], device=DEV)
    gone = (pages * bs >= st["lens"][1].long()[:, None]) & (table >= 0)
    ref.scatter_add_(0, table.long().clamp(min=0).flatten(), -gone.flatten().to(torch.int32))
    table.masked_fill_(gone, -1)
    return {"table": table, "lens": st["lens"][1], "ref": ref, "granted": st["granted"], "k": st["k"], "v": st["v"]}


def _plain_keep(st):
    case = st["case"]
    B, H, n, keep, bs = case["batch"], case["h_kv"], case["n"], _kept(case), case["block"]
    kept = torch.zeros((B, H, n), dtype=torch.bool, device=DEV).scatter_(-1, st["idx"].long(), True)
    slot = torch.arange(n, device=DEV)
    hole, fill = ((~kept & (slot < keep)).nonzero(as_tuple=True), (kept & (slot >= keep)).nonzero(as_tuple=True))
    where = slot.expand(B, H, n).clone()
    where[hole] = fill[2]
    for x in (st["k"], st["v"]):
        if bs:
            at = [(st["table"][y[0], y[2] // bs].long(), y[2] % bs, y[1]) for y in (hole, fill)]
            x[at[0]] = x[at[1]]
        else:
            x[hole] = x[fill]
    st["pos"][..., :keep] = where[..., :keep].to(torch.int32)
    st["acc"][..., :keep] = st["scores"].gather(-1, where)[..., :keep]
    st["lens"].copy_(st["counts"])
    st["seen"].fill_(n)
    return {x: st[x] for x in ("k", "v", "pos", "acc", "lens", "seen")}


def _plain_turn(case, x, pos, back):
    """Rows x [..., 128] turned by their positions pos [...]; 64-bit angles."""
    rot, half = case["rot"], case["rot"] // 2
    f, scale = _plain_frequencies(case)
    a = pos[..., None].double() * f
    c, s = (a.cos() * scale).float(), (a.sin() * scale).float()
    if back:
        s = -s
    x = x.float()
    y = x.clone()
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y.to(torch.bfloat16)


THETA, BEFORE = 500000.0, 8192       # base of the frequencies, and the context that a model was first trained on


def _plain_frequencies(case):
    """Angles per position of every pair, and the factor of the rotated values."""
    rot, kind, s = case["rot"], case["scaling"], case["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    theta = THETA * s ** (rot / (rot - 2)) if kind == "ntk" else THETA
    f, scale = theta ** (-2.0 * i / rot), 1.0
    if kind == "linear":
        f = f / s
    if kind == "yarn":
        low, high = (rot * math.log(BEFORE / (b * 2 * math.pi)) / (2 * math.log(THETA)) for b in (32.0, 1.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f, scale = f * (ramp / s + 1 - ramp), 0.1 * math.log(s) + 1
    if kind == "bands":
        turns = BEFORE * f / (2 * math.pi)
        f = f * (((turns - 1.0) / 3.0).clamp(0, 1) * (1 - 1 / s) + 1 / s)
    if case.get("direction", "inverse") == "inverse":
        scale = 1 / scale
    return f, scale


def _plain_rope(st):
    case = st["case"]
    hq, hk, back = case["h_q"], case["h_kv"], case["direction"] != "forward"
    y = _plain_turn(case, st["x"][:, :, :hq + hk], st["pos"][:, :, None], back).transpose(1, 2)
    return {"q": y[:, :hq].contiguous(), "k": y[:, hq:].contiguous()}


def _plain_unrope(st):
    case = st["case"]
    B, H, n = case["batch"], case["h_kv"], case["n"]
    x = st["key"]
    if case["block"]:
        x = x[st["table"].long()].reshape(B, -1, H, D)[:, :n].transpose(1, 2)
    return {"out": _plain_turn(case, x, st["pos"], True)}


# ------------------------------------------------------------------------------ the framework's calls
def _workspace(size):
    from kv_cache_eviction_window_gb300 import binding

    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    binding.kvsel_workspace_init(ws)
    return ws


def _own_tree(st):
    from kv_cache_eviction_window_gb300 import binding

    case = st["case"]
    if "plan" not in st:      # what a program keeps from step to step: parameters, cache view, workspace
        st["plan"] = binding.make_attn_params(h_kv=case["h_kv"], group=case["group"], batch=case["batch"], n_new=case["nodes"],
                                              max_len=case["len_max"], window=case["window"], n_sink=case["n_sink"])
        paged = case["cache"] == "paged"
        st["kv"] = binding.make_kv_paged(st["k"], st["v"], st["table"]) if paged else binding.make_kv_contiguous(st["k"], st["v"])
        st["ws"] = _workspace(binding.kvsel_attend_tree_workspace_size(st["plan"]))
    got = {}
    if case["masks"]:
        binding.kvsel_tree_masks(st["parents"], st["tree"], pos=st["pos"], first=st["first"], new_lens=st["new_lens"])
        got = {"tree": st["tree"], "pos": st["pos"]}
    binding.kvsel_attend_tree(st["plan"], st["q"], st["kv"], st["lens"], st["tree"], st["out"], st["ws"], new_lens=st["new_lens"], lse=st["lse"])
    return dict(got, out=st["out"], lse=st["lse"])


def _own_verify(st):
    from kv_cache_eviction_window_gb300 import binding

    case = st["case"]
    if "plan" not in st:
        st["plan"] = binding.make_verify_params(batch=case["batch"], n_new=case["nodes"], vocab=case["vocab"], mode=case["mode"], dtype=case["dtype"])
        st["ws"] = _workspace(binding.kvsel_verify_workspace_size(st["plan"]))
    binding.kvsel_verify(st["plan"], st["tokens"], st["parents"], st["target"], st["path"], st["counts"], st["next"], st["ws"], draft=st["draft"],
                         u=st["u"], new_lens=st["new_lens"])
    return {x: st[x] for x in ("path", "counts", "next")}


def _own_pool(st):
    from kv_cache_eviction_window_gb300 import binding

    case = st["case"]
    if "plan" not in st:
        st["plan"] = binding.make_pages_params(batch=case["batch"], max_blocks=st["table"][0].shape[1], num_blocks=st["k"].shape[1], block_size=case["block"],
                                               h_kv=case["h_kv"], layers=case["layers"], n_new=case["n_new"])
        st["ws"] = _workspace(binding.kvsel_pages_workspace_size(st["plan"]))
    return binding, st["plan"], st["ws"]


def _own_beam(st):
    binding, plan, ws = _own_pool(st)
    a = st["now"]
    st["now"] = 1 - a
    table, lens = st["table"][1 - a], st["lens"][1 - a]
    binding.kvsel_pages_fork(plan, st["table"][a], st["lens"][a], st["src"], table, lens, st["ref"], ws)
    binding.kvsel_pages_reserve(plan, st["k"], st["v"], table, st["ref"], lens, st["granted"], ws)
    return {"table": table, "lens": lens, "ref": st["ref"], "granted": st["granted"], "k": st["k"], "v": st["v"]}


def _own_accept(st):
    binding, plan, ws = _own_pool(st)
    table, lens = st["table"][0], st["lens"][1]
    binding.kvsel_pages_reserve(plan, st["k"], st["v"], table, st["ref"], st["lens"][0], st["granted"], ws)
    binding.kvsel_pages_accept(plan, st["k"], st["v"], table, st["all"], st["path"], st["counts"], lens, ws)
    binding.kvsel_pages_trim(plan, table, st["ref"], lens, ws)
    return {"table": table, "lens": lens, "ref": st["ref"], "granted": st["granted"], "k": st["k"], "v": st["v"]}


def _own_keep(st):
    from kv_cache_eviction_window_gb300 import binding

    case = st["case"]
    if "plan" not in st:
        st["plan"] = binding.make_params(h_kv=case["h_kv"], group=1, n_ctx=case["n"], window=32, n_ctx_per_req=[case["n"]] * case["batch"],
                                         n_sink=0, n_recent=0, budget_ratio=(_kept(case) + 0.5) / case["n"])
        st["kv"] = binding.make_kv_paged(st["k"], st["v"], st["table"]) if case["block"] else binding.make_kv_contiguous(st["k"], st["v"])
        st["ws"] = _workspace(256)
    binding.kvsel_compact_in_place(st["plan"], st["kv"], st["idx"], st["counts"], st["offsets"], st["lens"], st["seen"], st["pos"], st["ws"],
                                   scores=st["scores"], acc=st["acc"])
    return {x: st[x] for x in ("k", "v", "pos", "acc", "lens", "seen")}


def _own_angles(case):
    from kv_cache_eviction_window_gb300 import binding

    return binding.kvsel_rope_table(rot_dim=case["rot"], layout="interleaved" if case["interleaved"] else "half", theta=THETA, scaling=case["scaling"],
                                    factor=case["factor"], orig_len=BEFORE, direction=case.get("direction", "inverse"))


def _own_rope(st):
    from kv_cache_eviction_window_gb300 import binding

    case = st["case"]
    hq, hk = case["h_q"], case["h_kv"]
    if "plan" not in st:
        st["plan"] = _own_angles(case)
        x = st["x"].transpose(1, 2)
        st["xq"], st["xk"] = x[:, :hq], x[:, hq:hq + hk]
    binding.kvsel_rope(st["plan"], st["xq"], st["pos"], q_out=st["q"], k=st["xk"], k_out=st["k"])
    return {"q": st["q"], "k": st["k"]}


def _own_unrope(st):
    from kv_cache_eviction_window_gb300 import binding

    case = st["case"]
    if "plan" not in st:
        st["plan"] = _own_angles(case)
        st["kv"] = binding.make_kv_paged(st["key"], st["key"], st["table"]) if case["block"] else binding.make_kv_contiguous(st["key"], st["key"])
        st["ws"] = _workspace(256)
    binding.kvsel_rope_cache(st["plan"], st["kv"], st["lens"], st["pos"], st["ws"], out=st["out"])
    return {"out": st["out"]}


# ------------------------------------------------------------------------------ definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"tree": _exact_tree, "verify": _exact_verify, "beam": _exact_beam, "accept": _exact_accept, "keep": _exact_keep, "rope": _exact_rope,
            "unrope": _exact_unrope}[case["op"]](case, st)


def _exact_tree(case, st):
    B, H, G, m = case["batch"], case["h_kv"], case["group"], case["nodes"]
    lens, new = _sizes(case)
    out = torch.zeros((B, G * H, m, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, G * H, m), dtype=torch.float64, device=DEV)
    parents, pos = st["parents"].tolist(), st["pos"].clone()
    for b in range(B):
        n, fresh = lens[b], new[b]
        hidden = torch.zeros((fresh, n), dtype=torch.bool, device=DEV)
        hidden[:, n - fresh:] = True
        depth = []
        for t in range(fresh):
            u, steps = t, 0
            line = [t]
            while parents[b][u] >= 0:
                u, steps = parents[b][u], steps + 1
                line.append(u)
            hidden[t, torch.tensor([n - fresh + x for x in line], device=DEV)] = False
            depth.append(steps)
            gone = n - fresh + steps - case["window"]
            if case["window"] and gone >= case["n_sink"]:
                hidden[t, case["n_sink"]:min(gone + 1, n - fresh)] = True
        if case["masks"]:
            pos[b, :fresh] = _ints([n - fresh + x for x in depth])
        for h in range(H):
            if case["cache"] == "paged":
                pages = st["table"][b, :-(-n // case["block"])].long()
                k, v = (st[x][pages, :, h].reshape(-1, D)[:n].double() for x in "kv")
            else:
                k, v = (st[x][b, h, :n].double() for x in "kv")
            for g in range(G):
                e = st["q"][b, h * G + g, :fresh].double() @ k.T / math.sqrt(D)
                e[hidden] = -math.inf
                norm = torch.logsumexp(e, 1)
                out[b, h * G + g, :fresh] = torch.exp(e - norm[:, None]) @ v
                lse[b, h * G + g, :fresh] = norm
    got = {"tree": st["tree"], "pos": pos} if case["masks"] else {}
    return dict(got, out=out, lse=lse)


def _exact_verify(case, st):
    B, m, mode = case["batch"], case["nodes"], case["mode"]
    path = [[-1] * m for _ in range(B)]
    counts, nxt = [], []
    parents, tokens, u, new = (st[x].tolist() for x in ("parents", "tokens", "u", "new_lens"))
    for b in range(B):
        row = lambda x, t: st[x][b, t].double().cpu()   # noqa: E731
        at, line = 0, [0]
        while True:
            left = row("target", at)
            whole = 1.0
            step = None
            for c in (t for t in range(1, new[b]) if parents[b][t] == at):
                x = tokens[b][c]
                if mode == "greedy":
                    ok = int((left == left.max()).nonzero()[0]) == x
                else:
                    q = row("draft", at) if mode == "sampled" else None
                    ok = u[b][c] * (float(q[x]) if q is not None else 1.0) * whole < float(left[x])
                if ok:
                    step = c
                    break
                if mode == "sampled":
                    left = torch.clamp(left - whole * q, min=0)
                    whole = float(left.sum())
                elif mode == "point":
                    whole -= float(left[x])
                    left[x] = 0.0
            if step is None:
                break
            at = step
            line.append(at)
        if mode == "greedy":
            nxt.append(int((left == left.max()).nonzero()[0]))
        else:
            c = torch.cumsum(left if float(left.sum()) > 0 else row("target", at), 0)
            nxt.append(min(int(torch.searchsorted(c, u[b][0] * c[-1], right=True)), case["vocab"] - 1))
        path[b][:len(line)] = line
        counts.append(len(line))
    return {"path": _ints(path), "counts": _ints(counts), "next": _ints(nxt)}


def _exact_reserve(case, table, ref, lens, k, v):
    bs, granted = case["block"], []
    uses, jobs = list(ref), []
    for b, n in enumerate(lens):
        job = []
        for i in range(n // bs, -(-(n + case["n_new"]) // bs)):
            page = table[b][i]
            if page < 0:
                job.append((i, -1))
            elif uses[page] > 1:
                job.append((i, page))
                uses[page] -= 1
        jobs.append(job)
    free, asked = [p for p, r in enumerate(ref) if r == 0], 0
    have = len(free)
    for b, job in enumerate(jobs):
        asked += len(job)
        if job and asked > have:
            granted.append(0)
            continue
        for i, page in job:
            to = free.pop(0)
            if page >= 0:
                rows = min(bs, lens[b] - i * bs)
                k[:, to, :rows], v[:, to, :rows] = k[:, page, :rows], v[:, page, :rows]
                ref[page] -= 1
            table[b][i], ref[to] = to, 1
        granted.append(case["n_new"])
    return granted


def _exact_pages(table, lens, ref, granted, k, v):
    return {"table": _ints(table), "lens": _ints(lens), "ref": _ints(ref), "granted": _ints(granted), "k": k.double(), "v": v.double()}


def _exact_beam(case, st):
    k, v = st["k"], st["v"]
    old, lens, ref = st["table"][0].tolist(), st["lens"][0].tolist(), st["ref"].tolist()
    src = st["src"].tolist()
    table = [list(old[s]) for s in src]
    for by, rows in ((1, table), (-1, old)):
        for row in rows:
            for page in row:
                if page >= 0:
                    ref[page] += by
    lens = [lens[s] for s in src]
    granted = _exact_reserve(case, table, ref, lens, k, v)
    return _exact_pages(table, lens, ref, granted, k, v)


def _exact_accept(case, st):
    k, v, bs = st["k"], st["v"], case["block"]
    table, lens, ref = st["table"][0].tolist(), st["lens"][0].tolist(), st["ref"].tolist()
    granted = _exact_reserve(case, table, ref, lens, k, v)
    after = []
    for b, (path, count, n) in enumerate(zip(st["path"].tolist(), st["counts"].tolist(), st["all"].tolist())):
        base = n - case["n_new"]
        for i in range(count):
            (p, x), (q, y) = divmod(base + path[i], bs), divmod(base + i, bs)
            for pool in (k, v):
                pool[:, table[b][q], y] = pool[:, table[b][p], x].clone()
        after.append(base + count)
        for i in range(-(-after[b] // bs), len(table[b])):
            if table[b][i] >= 0:
                ref[table[b][i]] -= 1
                table[b][i] = -1
    return _exact_pages(table, after, ref, granted, k, v)


def _exact_keep(case, st):
    B, H, n, keep = case["batch"], case["h_kv"], case["n"], _kept(case)
    k, v, pos, acc = st["k"].clone(), st["v"].clone(), st["pos"], st["acc"].double()
    for b in range(B):
        for h in range(H):
            stay = set(st["idx"][b, h].tolist())
            holes = [i for i in range(keep) if i not in stay]
            fills = sorted(i for i in stay if i >= keep)
            rank = list(range(keep))
            for to, of in zip(holes, fills):
                rank[to] = of
            rank = torch.tensor(rank, device=DEV)
            for x, y in ((k, st["k"]), (v, st["v"])):
                if case["block"]:
                    bs = case["block"]
                    slot = torch.arange(keep, device=DEV)
                    x[st["table"][b, slot // bs].long(), slot % bs, h] = y[st["table"][b, rank // bs].long(), rank % bs, h]
                else:
                    x[b, h, :keep] = y[b, h, rank]
            pos[b, h, :keep] = rank.to(torch.int32)
            acc[b, h, :keep] = st["scores"][b, h, rank].double()
    return {"k": k.double(), "v": v.double(), "pos": pos, "acc": acc, "lens": _ints([[keep] * H] * B), "seen": _ints([[n] * H] * B)}


def _exact_turn(case, x, pos, sign):
    """x [..., 128] in 64 bits, pair by pair as complex numbers."""
    rot, kind, s, L = case["rot"], case["scaling"], case["factor"], float(BEFORE)
    y = x.double().clone()
    grow = 0.1 * math.log(s) + 1 if kind == "yarn" else 1.0
    if case.get("direction", "inverse") == "inverse":
        grow = 1 / grow
    for i in range(rot // 2):
        f = THETA ** (-2 * i / rot)
        if kind == "linear":
            f /= s
        elif kind == "ntk":
            f = (THETA * s ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif kind == "yarn":
            where = [rot / 2 * math.log(L / (2 * math.pi * b)) / math.log(THETA) for b in (32, 1)]
            low, high = max(0, math.floor(where[0])), min(rot - 1, math.ceil(where[1]))
            w = min(1.0, max(0.0, (i - low) / (high - low if high > low else 0.001)))
            f = (1 - w) * f + w * f / s
        elif kind == "bands":
            wave = 2 * math.pi / f
            if wave > L:
                f /= s
            elif wave > L / 4:
                w = (L / wave - 1) / 3
                f = (1 - w) * f / s + w * f
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
        z = torch.polar(torch.full(pos.shape, grow, dtype=torch.float64, device=DEV), sign * pos.double() * f)
        z = torch.complex(x[..., a].double(), x[..., b].double()) * z
        y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_rope(case, st):
    hq, hk = case["h_q"], case["h_kv"]
    sign = 1.0 if case["direction"] == "forward" else -1.0
    pos = st["pos"][:, None, :]
    return {name: _exact_turn(case, st["x"][:, :, a:a + h].transpose(1, 2), pos.expand(-1, h, -1), sign) for name, a, h in (("q", 0, hq), ("k", hq, hk))}


def _exact_unrope(case, st):
    B, H, n = case["batch"], case["h_kv"], case["n"]
    if not case["block"]:
        return {"out": _exact_turn(case, st["key"], st["pos"], -1.0)}
    out = torch.zeros((B, H, n, D), dtype=torch.float64, device=DEV)
    bs = case["block"]
    for b in range(B):
        row = torch.arange(n, device=DEV)
        page = st["table"][b, row // bs].long()
        for h in range(H):
            out[b, h] = _exact_turn(case, st["key"][page, row % bs, h], st["pos"][b, h], -1.0)
    return {"out": out}
