"""Helpers of the tests of kvsel_attend and kvsel_evict_append: build a cache in any layout with
unseen rows poisoned, run the call, and compare with the fp64 oracle under tolerances derived
from the roundings that the kernels make.  Importing this module does not need a GPU."""
import numpy as np

from oracle import cache_oracle as CO

D = 128
NAN = 0x7FC0          # bf16 bit pattern of a NaN


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def bf16(x):
    """float array -> nearest bf16 values, as float64 (ties to even)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) >> 16
    return (u.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bits(x):
    """bf16 values (float64) -> bit patterns; NaN stays NaN."""
    return (np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def to_gpu_bf16(x):
    import torch

    return torch.from_numpy(bits(x).view(np.int16)).cuda().view(torch.bfloat16)


def to_f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Case:
    """One call: lens [B][H] rows, new [B] tokens, all values in bf16."""

    def __init__(self, *, B=1, H=2, G=4, m=1, lens=100, new=None, layout="contiguous", block=16, window=0, n_sink=0,
                 causal=True, per_head=False, token_major=False, scale=0.0, seed=0, logit=1.5, pad_rows=0):
        g = rng(seed)
        self.__dict__.update(B=B, H=H, G=G, m=m, layout=layout, block=block, window=window, n_sink=n_sink,
                             causal=causal, per_head=per_head, token_major=token_major, scale=scale)
        lens = np.broadcast_to(np.asarray(lens), (B, H) if per_head or layout == "packed" else (B,))
        self.lens = (lens if lens.ndim == 2 else np.repeat(lens[:, None], H, 1)).astype(int)
        self.new = np.full(B, m) if new is None else np.asarray(new, int)
        self.new_given = new is not None
        self.max_len = max(1, int(self.lens.max())) + pad_rows
        self.q = bf16(g.standard_normal((B, H, G, m, D)) * logit)
        self.k = [[bf16(g.standard_normal((n, D)) * np.exp(0.5 * g.standard_normal((n, 1)))) for n in r] for r in self.lens]
        self.v = [[bf16(g.standard_normal((n, D))) for n in r] for r in self.lens]
        self.g = g

    def seen_rows(self, b, h):
        n, m = self.lens[b][h], self.new[b]
        return CO.visible(n, m, self.causal, self.window, self.n_sink).any(axis=0) if m else np.zeros(n, bool)

    def oracle(self):
        kw = dict(causal=self.causal, window=self.window, n_sink=self.n_sink, scale=self.scale or None)
        return [[CO.attend_segment(self.q[b, h, :, :self.new[b]], self.k[b][h], self.v[b][h], **kw)
                 for h in range(self.H)] for b in range(self.B)]

    # ---------------------------------------------------------------- device side
    def upload(self):
        import torch

        from kv_cache_eviction_window_gb300 import binding as L

        B, H, G, m = self.B, self.H, self.G, self.m
        ks, vs = [[None] * H for _ in range(B)], [[None] * H for _ in range(B)]
        for b in range(B):
            for h in range(H):
                see = self.seen_rows(b, h)[:, None]
                ks[b][h] = np.where(see, self.k[b][h], np.nan)
                vs[b][h] = np.where(see, self.v[b][h], np.nan)
        self.offsets = None
        if self.layout == "paged":
            bs = self.block
            nb = -(-self.max_len // bs)
            table = self.g.permutation(B * nb).reshape(B, nb).astype(np.int32)
            pool = [np.full((B * nb, bs, H, D), np.nan) for _ in range(2)]
            for b in range(B):
                used = np.zeros(nb * bs, bool)
                for h in range(H):
                    n = self.lens[b][h]
                    for x, src in zip(pool, (ks, vs)):
                        rows = np.full((nb * bs, D), np.nan)
                        rows[:n] = src[b][h]
                        x[table[b], :, h] = rows.reshape(nb, bs, D)
                    used[:n] |= self.seen_rows(b, h)
                # pages without a visible row may be gone
                table[b, ~used.reshape(nb, bs).any(axis=1)] = -1
            kt, vt = to_gpu_bf16(pool[0]), to_gpu_bf16(pool[1])
            tt = torch.from_numpy(table).cuda()
            self.keep = (kt, vt, tt)
            kv = L.make_kv_paged(kt, vt, tt)
        elif self.layout == "packed":
            flat = [(b, h) for b in range(B) for h in range(H)]
            off = np.cumsum([0] + [self.lens[b][h] for b, h in flat])
            self.n_rows = max(1, int(off[-1]))
            pad = [np.full((1 if off[-1] == 0 else 0, D), np.nan)]
            kt = to_gpu_bf16(np.concatenate([ks[b][h] for b, h in flat] + pad))
            vt = to_gpu_bf16(np.concatenate([vs[b][h] for b, h in flat] + pad))
            self.offsets = torch.from_numpy(off[:-1].astype(np.int64)).cuda()
            self.keep = (kt, vt)
            kv = L.make_kv_packed(kt, vt)
        else:
            # rows one line further apart than they are long, heads and requests with slack
            mem = [np.full((B, H, self.max_len, D + 8), np.nan) for _ in range(2)]
            for b in range(B):
                for h in range(H):
                    for x, src in zip(mem, (ks, vs)):
                        x[b, h, :self.lens[b][h], :D] = src[b][h]
            kt, vt = (to_gpu_bf16(x)[..., :D] for x in mem)
            self.keep = (kt, vt)
            kv = L.make_kv_contiguous(kt, vt)
        if self.token_major:
            wide = to_gpu_bf16(np.full((B, m, (G + 2) * H, D), np.nan))
            qt = wide[:, :, :G * H].permute(0, 2, 1, 3)
            qt.copy_(to_gpu_bf16(self.q.reshape(B, H * G, m, D)))
            out = to_gpu_bf16(np.full((B, m, G * H, D), 7.0)).permute(0, 2, 1, 3)
            qs, os_ = qt.stride()[:3], out.stride()[:3]
        else:
            qt = to_gpu_bf16(self.q.reshape(B, H * G, m, D))
            out = to_gpu_bf16(np.full((B, G * H, m, D), 7.0))
            qs = os_ = (0, 0, 0)
        self.params = dict(h_kv=H, group=G, batch=B, n_new=m, max_len=self.max_len, causal=self.causal, window=self.window,
                           n_sink=self.n_sink, scale=self.scale, lens_per_head=self.per_head, q_strides=qs, o_strides=os_,
                           n_rows=self.n_rows if self.layout == "packed" else 0, acc_stride=self.max_len + 3)
        lens = self.lens if self.per_head or self.layout == "packed" else self.lens[:, 0]
        self.t = dict(q=qt, kv=kv, out=out, lens=torch.from_numpy(np.ascontiguousarray(lens, np.int32)).cuda(),
                      new_lens=torch.from_numpy(self.new.astype(np.int32)).cuda() if self.new_given else None,
                      lse=torch.full((B, G * H, m), 7.0, device="cuda"),
                      acc=torch.zeros((B, H, self.max_len + 3), device="cuda"))
        return self

    def call(self, acc=False, ws=None, stream=None, lse=True):
        from kv_cache_eviction_window_gb300 import binding as L

        p = L.make_attn_params(**self.params)
        if ws is None:
            ws = workspace(L.kvsel_attend_workspace_size(p, acc))
        t = self.t
        L.kvsel_attend(p, t["q"], t["kv"], t["lens"], t["out"], ws, new_lens=t["new_lens"], offsets=self.offsets,
                       lse=t["lse"] if lse else None, acc=t["acc"] if acc else None, stream=stream)
        return ws

    def check(self, ora=None, acc=False, calls=1):
        """Compare the device results with the oracle's.

        u = 2^-23 bounds one fp32 operation (the tensor cores may cut instead of round).  A logit is a
        sum of d exact products: off by e = (d + 4) u * max sum |q||k| scale, the exponential's argument
        and its result by a few u more (the argument is at most a few hundred: 2^-14 covers it).  The
        softmax weights are off by 2 e' relative, e' = e + 2^-14, and by a bf16 rounding, 2^-8, where
        the second product takes them in bf16; out by that times sum w |v|, and rounded to bf16."""
        ora = ora or self.oracle()
        B, H, G, m = self.B, self.H, self.G, self.m
        out = to_f64(self.t["out"]).reshape(B, H, G, m, D)
        lse = self.t["lse"].cpu().numpy().astype(np.float64).reshape(B, H, G, m)
        got = self.t["acc"].cpu().numpy().astype(np.float64)
        for b in range(B):
            for h in range(H):
                o, mb, n = ora[b][h], self.new[b], self.lens[b][h]
                e = (D + 4) * 2.0 ** -23 * o["abs_logit"] + 2.0 ** -14
                tol = (2 * e[..., None] + 2.0 ** -8) * o["mean_abs"] + 2.0 ** -8 * np.abs(o["out"]) + 1e-30
                err = np.abs(out[b, h, :, :mb] - o["out"])
                assert np.all(err <= tol), (b, h, float(np.nanmax(err / tol)), np.isnan(err).sum())
                want = o["lse"]
                fin = np.isfinite(want)
                assert np.array_equal(np.isneginf(lse[b, h, :, :mb]), ~fin), (b, h)
                le = np.abs(lse[b, h, :, :mb][fin] - want[fin])
                assert np.all(le <= e[fin] + 2.0 ** -21 * np.abs(want[fin])), (b, h, float(le.max()))
                # rows behind the request's tokens stay as they were
                assert np.all(out[b, h, :, mb:] == 7.0) and np.all(lse[b, h, :, mb:] == 7.0)
                if acc:
                    w = calls * o["weight"]
                    et = (2 * e.max(initial=0.0) + (G * mb + 2) * 2.0 ** -23) * w + 1e-30
                    d = np.abs(got[b, h, :n] - w)
                    assert np.all(d <= et), (b, h, float((d / et).max()))
                    assert np.all(got[b, h, n:] == 0.0)


def token_tolerance(o, n):
    """How far a row of the kernel of few rows may be from the oracle's o (n cached rows).

    A logit is off by e = (D + 4) 2^-23 max sum |q||k| scale as above; in the exponent's argument it is rounded
    twice, |argument| <= 3 abs_logit in log2 units, and ex2.approx is off by 2^-22: weights are off by 2 e'
    (over their sum).  They enter the second product as a bf16 part and a bf16 remainder, each off by at most
    half a step, 2^-8: 2^-16 in all.  A warp adds two products for each of its at most n / 4 + 16 rows, and as
    many weights into the sum; rescaling and joining parts add less than a hundred roundings more: (n + 128)
    2^-23.  The result is rounded once to bf16, 2^-8."""
    e = (D + 4) * 2.0 ** -23 * o["abs_logit"] + (3 * o["abs_logit"] + 4) * 2.0 ** -22
    w = 2 * e[..., None] + 2.0 ** -16 + (n + 128) * 2.0 ** -23
    return w * (1 + 2.0 ** -8) * o["mean_abs"] + 2.0 ** -8 * np.abs(o["out"]) + 1e-30


def paired(c):
    """Values in pairs of opposite rows, so that results are small next to what they are summed from: a rounding
    of the weights shows, the rounding of the result does not."""
    for r in c.v:
        for v in r:
            v[1::2] = -v[:v.shape[0] // 2 * 2:2]
    return c


def marked(c):
    """Values that name their rows: column u of 64 is non-zero in every 64th unit of 16 rows, the others in
    every 64th row, so with even weights a unit that is lost, read twice or misplaced moves its column by a
    few per cent at 20,000 rows, and by more at fewer."""
    for r in c.v:
        for v in r:
            j = np.arange(v.shape[0])
            v[:] = 0.0
            v[j, j // 16 % 64] = 1.0 + j // 1024 % 4
            v[j, 64 + j % 64] = 1.0 + j // 64 % 4
    return c


def check_tokens(c, ora=None):
    """Results of the kernel of few rows under its own bound (rows of every token of a request)."""
    ora = ora or c.oracle()
    out = to_f64(c.t["out"]).reshape(c.B, c.H, c.G, c.m, D)
    for b in range(c.B):
        for h in range(c.H):
            o, mb = ora[b][h], c.new[b]
            tol = token_tolerance(o, c.lens[b][h])
            err = np.abs(out[b, h, :, :mb] - o["out"])
            assert np.all(err <= tol), (b, h, float(np.nanmax(err / tol)), np.isnan(err).sum())


def workspace(nbytes):
    import torch

    from kv_cache_eviction_window_gb300 import binding as L

    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    # what an earlier call may have left there
    ws[256 + 65536:].fill_(0xFF)
    L.kvsel_workspace_init(ws)
    return ws


def status(ws):
    import torch

    from kv_cache_eviction_window_gb300 import binding as L

    torch.cuda.synchronize()
    return L.kvsel_get_device_status(ws)
