"""Seeded caches, tables and bounds of error that the GPU tests of the long-context operators share."""
import numpy as np
import torch

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f8": torch.float8_e4m3fn, "f32": torch.float32}
EDGES = [1, 0, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400, -3]


def i32(a, device):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=device)


def n64(t):
    return t.detach().float().double().cpu().numpy()


class Paged:
    """Requests of the given lengths in one paged cache; rows that no request holds are NaN."""

    def __init__(self, device, seed, lens, Hk, d, cache, ps, layout="nhd", cols=None, spare=3, nan=True):
        rng = self.rng = np.random.default_rng(seed)
        self.device, self.cache, self.ps, self.Hk, self.d, self.layout = device, cache, ps, Hk, d, layout
        self.lens = np.asarray(lens)
        have = -(-np.maximum(self.lens, 0) // ps)
        cols = cols or max(1, int(have.max()))
        have = np.minimum(have, cols)
        self.pages = int(have.sum()) + spare
        self.table = np.full((len(lens), cols), -1)
        self.table[np.arange(cols)[None] < have[:, None]] = rng.permutation(self.pages)[:have.sum()]
        self.scale = 0.03125 if cache == "f8" else 1.0
        self.k, self.v = (self.make(nan) for _ in range(2))

    def used(self):
        got = np.zeros((self.pages, self.ps), bool)
        for r, n in enumerate(self.lens):
            j = np.arange(min(max(int(n), 0), self.table.shape[1] * self.ps))
            p = self.table[r, j // self.ps]
            ok = (p >= 0) & (p < self.pages)
            got[p[ok], j[ok] % self.ps] = True
        return got

    def make(self, nan):
        c = torch.tensor(self.rng.standard_normal((self.pages, self.ps, self.Hk, self.d)) / self.scale, dtype=torch.float32)
        if nan:
            c[torch.tensor(~self.used())] = float("nan")
        c = c.to(TYPES[self.cache])
        if self.layout == "hnd":
            t = c.dtype
            c = c.view(torch.uint8 if self.cache == "f8" else t).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3).view(t)
        return c.to(self.device)

    def queries(self, *shape):
        q = torch.tensor(self.rng.standard_normal(shape), device=self.device)
        return q.to(torch.float32 if self.cache == "f32" else torch.bfloat16)

    def t(self, a):
        return i32(a, self.device)

    def k64(self):
        return n64(self.k) * self.scale

    def v64(self):
        return n64(self.v) * self.scale


def spread(q, k, scale):
    """D of one query and its keys: how far a score may be off.  A score is a sum of d products (exact in fp32 for
    bf16 and 8-bit values) with at most d roundings, so within (d + 4) u of scale * sum |q k|; as the exponent of 2
    it is rounded twice more, 2 u |s| in all."""
    return ((len(q) + 6) * U * abs(scale) * (np.abs(k) @ np.abs(q)).max()) if len(k) else 0.0


def attention_bound(q, k, v, want, scale, bf16, weights, lse=0.0):
    """(bound of o, bound of lse) of one query head.  Every exponential is within 2 D + 4 u of itself, their sum within
    n u more for n tokens; `weights` is what else a weight may be off by, and a part of the tokens that is joined by
    its lse (fp32) is off by 4 u (1 + |lse|) more.  The quotient is a weighted mean of v, so its error is at most twice
    that of the weights times the largest |v|, and the output's own rounding 2^-8 |o| (bf16) or u |o|."""
    w = 2 * spread(q, k, scale) + 4 * U + len(k) * U + weights + 4 * U * (1 + abs(lse))
    return 2 * w * np.abs(v).max() + (2.0 ** -8 if bf16 else U) * np.abs(want), w + 4 * U * abs(lse)


def compare(got, want, rows_of, q, scale, bf16, weights):
    """Worst ratios of error and bound of (o, lse); rows_of(r, h) gives the keys and values that head h of row r
    attends to."""
    o, lse, q = n64(got[0]), n64(got[1]), n64(q)
    assert np.isfinite(o).all()
    np.testing.assert_array_equal(np.isneginf(lse), np.isneginf(want[1]))
    worst = [0.0, 0.0]
    for r in range(o.shape[0]):
        for h in range(o.shape[1]):
            k, v = rows_of(r, h)
            if len(k) == 0:
                assert (o[r, h] == 0).all() and lse[r, h] == -np.inf
                continue
            bo, bl = attention_bound(q[r, h], k, v, want[0][r, h], scale, bf16, weights, want[1][r, h])
            worst[0] = max(worst[0], float((np.abs(o[r, h] - want[0][r, h]) / bo).max()))
            worst[1] = max(worst[1], abs(lse[r, h] - want[1][r, h]) / bl)
    return worst


def ratios(got, want, rows_of, q, scale, bf16, weights):
    """Ratios of error and bound of o (rows, heads, d) and of lse (rows, heads), as `compare` bounds them; inf where a
    result is NaN or infinite and should not be, and where a query without tokens has anything but o = 0 and lse = -inf."""
    o, lse, q = n64(got[0]), n64(got[1]), n64(q)
    ro, rl = np.full(o.shape, np.inf), np.full(lse.shape, np.inf)
    for r in range(o.shape[0]):
        for h in range(o.shape[1]):
            k, v = rows_of(r, h)
            if len(k) == 0:
                ro[r, h], rl[r, h] = np.where(o[r, h] == 0, 0.0, np.inf), 0.0 if lse[r, h] == -np.inf else np.inf
                continue
            bo, bl = attention_bound(q[r, h], k, v, want[0][r, h], scale, bf16, weights, want[1][r, h])
            ro[r, h], rl[r, h] = np.abs(o[r, h] - want[0][r, h]) / bo, abs(lse[r, h] - want[1][r, h]) / bl
    return np.where(np.isnan(ro), np.inf, ro), np.where(np.isnan(rl), np.inf, rl)


def attended(s):
    """rows_of of `ratios` for rows behind shared prefixes (test_prefix_attn_gpu.Shared)."""
    from oracle.longctx import _tokens
    k64, v64, at = s.k64(), s.v64(), []
    for r, p in enumerate(s.prefix):
        t = _tokens(s.ptable[p], s.plens[p], s.ps, s.pages) if 0 <= p < len(s.plens) else []
        t = t + _tokens(s.own[r], s.rows[r], s.ps, s.pages)
        at.append((np.array([x[1] for x in t], int), np.array([x[2] for x in t], int)))
    return lambda r, h: (k64[(*at[r], h * s.Hk // s.H)], v64[(*at[r], h * s.Hk // s.H)])


def captured(call):
    """`call` run once on a side stream and then captured; the graph."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g
