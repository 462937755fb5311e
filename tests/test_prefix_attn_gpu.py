"""ssm_prefix_attn_decode_fwd on the GPU against the fp64 oracle; the bounds are derived in
longctx_cases.attention_bound, with 2^-17 for softmax weights that enter their product as two bf16
values."""
import numpy as np
import pytest

from helpers import lib, report
from longctx_cases import EDGES, Paged, captured, compare, n64
from oracle import longctx

pytestmark = pytest.mark.gpu


class Shared(Paged):
    """Rows of own lengths behind prefixes of other lengths, in one cache: the first lens are the rows'."""

    def __init__(self, device, seed, plens, prefix, lens, H, Hk, d, cache, ps, layout="nhd", **kw):
        super().__init__(device, seed, list(lens) + list(plens), Hk, d, cache, ps, layout, **kw)
        n = len(lens)
        self.H, self.plens, self.prefix = H, np.asarray(plens), np.asarray(prefix)
        self.own, self.ptable, self.rows = self.table[:n].copy(), self.table[n:].copy(), self.lens[:n]
        self.q = self.queries(n, H, d)
        self.sc = d ** -0.5

    def call(self, **kw):
        return lib().ssm_prefix_attn_decode_fwd(self.q, self.k, self.v, self.t(self.prefix), self.t(self.ptable), self.t(self.plens),
                                                self.t(self.own), self.t(self.rows), scale=self.sc, k_scale=self.scale,
                                                v_scale=self.scale, return_lse=True, **kw)

    def want(self):
        return longctx.prefix_attn_decode(n64(self.q), self.k64(), self.v64(), self.prefix, self.ptable, self.plens, self.own,
                                          self.rows, self.sc)

    def check(self, name, got=None):
        got, want, k64, v64 = got or self.call(), self.want(), self.k64(), self.v64()
        cache = {}

        def tokens(r):
            if r not in cache:
                p = self.prefix[r]
                t = longctx._tokens(self.ptable[p], self.plens[p], self.ps, self.pages) if 0 <= p < len(self.plens) else []
                t = t + longctx._tokens(self.own[r], self.rows[r], self.ps, self.pages)
                cache[r] = np.array([x[1] for x in t], int), np.array([x[2] for x in t], int)
            return cache[r]

        def rows_of(r, h):
            g = h * self.Hk // self.H
            return k64[(*tokens(r), g)], v64[(*tokens(r), g)]

        bf = self.cache != "f32"
        worst = compare(got, want, rows_of, self.q, self.sc, bf, 2.0 ** -17 if bf else 0.0)
        report("prefix " + name, o_of_bound=worst[0], lse_of_bound=worst[1])
        assert worst[0] <= 1.0 and worst[1] <= 1.0, worst
        return got


CASES = [  # prefix lengths, prefix of each row, own lengths, H, Hk, d, cache, page, layout
    ([300], [0] * 4, [5, 0, 17, 64], 4, 2, 64, "bf16", 16, "nhd"),
    ([129], [0], [3], 1, 1, 64, "bf16", 16, "nhd"),
    ([1], [0], [0], 2, 1, 128, "bf16", 1, "nhd"),
    ([700], [0] * 20, EDGES, 8, 2, 128, "bf16", 16, "nhd"),
    ([700, 33, 0, 257], [0] * 7 + [1] * 3 + [-1, 9] + [2] * 3 + [3] * 5, EDGES, 6, 2, 128, "bf16", 8, "hnd"),
    ([100, 200, 300], [i % 3 for i in range(20)], EDGES, 5, 1, 80, "bf16", 24, "nhd"),       # rows in any order
    ([511], [0] * 20, EDGES, 4, 4, 96, "bf16", 7, "hnd"),
    ([257, 65], [0] * 11 + [1] * 9, EDGES, 2, 2, 192, "bf16", 64, "nhd"),
    ([385], [0] * 20, EDGES, 4, 1, 256, "bf16", 16, "nhd"),
    ([200], [0] * 3, [9, 0, 40], 17, 1, 128, "bf16", 16, "nhd"),
    ([200, 50], [0, 1, 0], [9, 0, 40], 70, 1, 64, "bf16", 16, "nhd"),                         # more heads than a block's columns
    ([200, 50], [0, 1, 0], [9, 0, 40], 80, 2, 256, "bf16", 16, "nhd"),
    ([90], [0] * 20, EDGES, 3, 1, 8, "bf16", 5, "nhd"),
    ([600], [0] * 20, EDGES, 8, 2, 128, "f8", 16, "nhd"),
    ([1000, 100], [0] * 10 + [1] * 10, EDGES, 8, 1, 64, "f8", 64, "hnd"),
    ([333], [0] * 20, EDGES, 5, 1, 96, "f8", 24, "hnd"),
    ([333], [0] * 20, EDGES, 4, 2, 192, "f8", 1, "nhd"),
    ([129, 128], [1, 0] * 10, EDGES, 2, 1, 256, "f8", 8, "nhd"),
    ([129], [0] * 20, EDGES, 6, 2, 16, "f8", 16, "nhd"),
    ([333], [0] * 20, EDGES, 5, 1, 256, "f32", 24, "nhd"),
    ([200, 70], [0] * 12 + [1] * 8, EDGES, 4, 4, 128, "f32", 16, "hnd"),
    ([150], [0] * 20, EDGES, 20, 1, 64, "f32", 8, "nhd"),
    ([64], [0] * 20, EDGES, 3, 3, 192, "f32", 1, "nhd"),
    ([333], [0] * 20, EDGES, 2, 1, 72, "f32", 16, "nhd"),
    ([9001], [0] * 3, [100, 0, 7], 4, 1, 64, "bf16", 64, "hnd"),                              # one prefix over every block
    ([5000], [0] * 64, list(range(64)), 8, 2, 128, "bf16", 16, "nhd"),
    ([64, 64, 64, 64, 64], [i // 30 for i in range(150)], [i % 5 for i in range(150)], 2, 2, 64, "bf16", 16, "nhd"),
    ([40], [0] * 300, [1] * 300, 4, 4, 64, "f32", 16, "nhd"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%d-%d-%d-H%d-%d-d%d-%s-p%d-%s" % ((max(c[0]), len(c[0]), len(c[2])) + c[3:]))
def test_against_the_oracle(cuda_device, case):
    Shared(cuda_device, 40 + case[5], *case).check(str(case[3:]))


def test_scores_of_every_size(cuda_device):
    """Scores of hundreds of either sign, and equal ones."""
    for sc in (8.0, -8.0, 0.0):
        s = Shared(cuda_device, 51, [300], [0] * 5, [40, 0, 3, 64, 1], 4, 2, 64, "f32", 16)
        s.sc = sc
        s.check("scale %g" % sc)
        s = Shared(cuda_device, 52, [300], [0] * 5, [40, 0, 3, 64, 1], 4, 2, 64, "bf16", 16)
        s.sc = sc / 4
        s.check("bf16 scale %g" % sc)


def test_maxima_that_rise(cuda_device):
    """Keys along the query that grow from tile to tile: the running maximum is raised again and again, by less and by
    more than the slack that it is given."""
    import torch
    for step in (0.002, 0.02, 0.2):
        s = Shared(cuda_device, 53, [2000], [0] * 3, [5, 0, 1], 2, 1, 64, "f32", 16)
        j = np.arange(2000)
        s.q[:] = 1.0
        k = torch.tensor(np.random.default_rng(1).standard_normal((2000, 64)) * 0.1 + (j * step)[:, None] / 64, dtype=torch.float32)
        s.k[torch.tensor(s.ptable[0][j // 16]), torch.tensor(j % 16), 0] = k.to(cuda_device)
        s.sc = 1.0
        s.check("rising %g" % step)


def test_infinite_and_nan_keys(cuda_device):
    """-inf scores weigh nothing, in the prefix and in a row's own tokens; a row of only those is empty; a NaN key of
    the prefix reaches every row that shares it and no other."""
    s = Shared(cuda_device, 54, [40, 40, 40], [0, 1, 2, -1], [0, 0, 3, 4], 2, 1, 64, "f32", 16)
    s.q = s.q.abs() + 0.1
    at = lambda p, j: (int(s.ptable[p, j // 16]), j % 16)  # noqa: E731
    for j in range(3, 20):
        s.k[at(0, j)][0, 5] = -float("inf")
    for j in range(40):
        s.k[at(1, j)][0, 7] = -float("inf")
    s.k[at(2, 11)][0, 0] = float("nan")
    o, lse = s.call()
    import torch
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    assert o[2].isnan().all() and lse[2].isnan().all()
    assert o[[0, 3]].isfinite().all() and lse[[0, 3]].isfinite().all()
    keep = [j for j in range(40) if not 3 <= j < 20]
    k, v = (torch.stack([c[at(0, j)][0] for j in keep]).double() for c in (s.k, s.v))
    sc = s.sc * s.q[0].double() @ k.T
    # 23 scores of about 20: within 1e-5 by the bounds
    assert (o[0].double() - torch.softmax(sc, -1) @ v).abs().max() <= 2e-4
    assert (lse[0].double() - torch.logsumexp(sc, -1)).abs().max() <= 2e-4


def test_bad_pages_long_lengths_and_given_tensors(cuda_device):
    """Pages outside the cache hold no token, lengths end with their table, q and both tables are strided, and o, lse and
    a workspace that holds NaN are the caller's."""
    import torch
    m = lib()
    s = Shared(cuda_device, 55, [200, 90], [0, 0, 1, 0, 1], [70, 0, 33, 5, 16], 6, 2, 128, "bf16", 16)
    s.ptable[0, 3], s.ptable[0, 5], s.ptable[1, 0], s.own[0, 1] = -1, s.pages, 1 << 30, -7
    cols = s.own.shape[1]
    big = torch.full((5, cols + 4), -1, dtype=torch.int32, device=cuda_device)
    big[:, :cols] = s.t(s.own)
    pbig = torch.full((2, s.ptable.shape[1] + 3), -1, dtype=torch.int32, device=cuda_device)
    pbig[:, :s.ptable.shape[1]] = s.t(s.ptable)
    proj = torch.randn((5, 2048), device=cuda_device).to(torch.bfloat16)
    s.q = proj[:, 256:1024].view(5, 6, 128)
    s.plens, s.rows = np.array([1 << 20, 90]), np.array([1 << 30, 0, 33, 5, 16])
    ws = torch.full((m.ssm_prefix_attn_decode_fwd_workspace_size(5, 6, 2, 128, s.ptable.shape[1], cols, 16),), 255, dtype=torch.uint8,
                    device=cuda_device)
    o, lse = torch.empty((5, 6, 128), dtype=torch.bfloat16, device=cuda_device), torch.empty((5, 6), device=cuda_device)
    # what no request held before is read now: a number
    s.k, s.v = (torch.nan_to_num(c, nan=0.5) for c in (s.k, s.v))
    got = m.ssm_prefix_attn_decode_fwd(s.q, s.k, s.v, s.t(s.prefix), pbig[:, :s.ptable.shape[1]], s.t(s.plens), big[:, :cols], s.t(s.rows),
                                       scale=s.sc, o=o, lse=lse, workspace=ws)
    assert got[0].data_ptr() == o.data_ptr() and got[1].data_ptr() == lse.data_ptr()
    s.check("bad pages", got)


def test_the_same_as_pages_in_the_rows_own_tables(cuda_device):
    """Against ssm_paged_attn_decode_fwd with the prefix's pages in front of each row's own: the same tokens."""
    m = lib()
    s = Shared(cuda_device, 56, [320], [0] * 9, list(range(0, 90, 10)), 8, 2, 128, "bf16", 16)
    a = s.call()
    joined = np.concatenate([np.repeat(s.ptable[:, :20], 9, 0), s.own], 1)
    b = m.ssm_paged_attn_decode_fwd(s.q, s.k, s.v, s.t(joined), s.t(s.rows + 320), scale=s.sc, return_lse=True)
    # each is within half of a bf16 step and its weights' error of the exact value
    assert (np.abs(n64(a[0]) - n64(b[0])) <= 2.0 ** -7 * np.abs(n64(b[0])) + 1e-4).all()
    assert np.abs(n64(a[1]) - n64(b[1])).max() <= 1e-4


def test_twice_the_same_no_lse_and_another_stream(cuda_device):
    import torch
    s = Shared(cuda_device, 57, [3000, 100], [0] * 5 + [1] * 4, [9] * 9, 8, 2, 128, "f8", 64, "hnd")
    a, b = s.call(), s.call()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        c = s.call()
    other.synchronize()
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    o = lib().ssm_prefix_attn_decode_fwd(s.q, s.k, s.v, s.t(s.prefix), s.t(s.ptable), s.t(s.plens), s.t(s.own), s.t(s.rows), scale=s.sc,
                                         k_scale=s.scale, v_scale=s.scale)
    assert torch.equal(o, a[0])


def test_no_rows(cuda_device):
    import torch
    q = torch.zeros((0, 4, 64), device=cuda_device)
    c = torch.zeros((2, 16, 2, 64), device=cuda_device)
    i = lambda *n: torch.zeros(n, dtype=torch.int32, device=cuda_device)  # noqa: E731
    o, lse = lib().ssm_prefix_attn_decode_fwd(q, c, c.clone(), i(0), i(1, 2), i(1), i(0, 3), i(0), scale=1.0, return_lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_in_a_graph_with_everything_changing(cuda_device):
    """Captured once; q, the rows' prefixes and all lengths change in place between replays, with eager calls between
    them: every replay equals the eager call."""
    import torch
    m = lib()
    s = Shared(cuda_device, 58, [600, 300], [0, 0, 1, 1, 0], [60, 20, 33, 1, 0], 8, 2, 128, "bf16", 16, nan=False)
    prefix, plens, rows, own, pt = s.t(s.prefix), s.t(s.plens), s.t(s.rows), s.t(np.maximum(s.own, 0)), s.t(np.maximum(s.ptable, 0))
    o, lse = torch.empty_like(s.q), torch.empty((5, 8), device=cuda_device)
    ws = torch.empty(m.ssm_prefix_attn_decode_fwd_workspace_size(5, 8, 2, 128, pt.shape[1], own.shape[1], 16), dtype=torch.uint8,
                     device=cuda_device)
    call = lambda: m.ssm_prefix_attn_decode_fwd(s.q, s.k, s.v, prefix, pt, plens, own, rows, scale=0.09, o=o, lse=lse, workspace=ws)  # noqa: E731
    g = captured(call)
    for ids, pl, n in (([0, 0, 1, 1, 0], [600, 300], [60, 20, 33, 1, 0]), ([1, 0, 1, 0, 5], [17, 300], [0, 0, 33, 1, 64]),
                       ([0] * 5, [0, 0], [0, 1, 2, 3, 4]), ([-1] * 5, [5, 5], [0] * 5), ([1] * 5, [0, 608], [64] * 5)):
        for t, v in ((prefix, ids), (plens, pl), (rows, n)):
            t.copy_(torch.tensor(v))
        s.q.copy_(torch.randn_like(s.q))
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        a, b = o.clone(), lse.clone()
        o.fill_(9.0)
        call()
        torch.cuda.synchronize()
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_a_prefix_past_4_gib(cuda_device):
    """Offsets past 32 bits: a prefix's pages at the end of a cache of 5 GiB a tensor."""
    import torch
    P, ps, Hk, d = 163840, 16, 8, 128
    s = Shared(cuda_device, 59, [77], [0, 0], [3, 16], 16, Hk, d, "bf16", ps)
    last = [P - 1, P - 40000, P - 3, 131072, 131071]
    big = [torch.zeros((P, ps, Hk, d), dtype=torch.bfloat16, device=cuda_device) for _ in range(2)]
    map_ = {int(p): q for p, q in zip(s.ptable[0, :5], last)}
    map_.update({int(s.own[r, 0]): 150000 + r for r in range(2)})
    for c, to in ((s.k, big[0]), (s.v, big[1])):
        for p, q in map_.items():
            to[q] = c[p]
    got = lib().ssm_prefix_attn_decode_fwd(s.q, big[0], big[1], s.t([0, 0]), s.t([last]), s.t([77]), s.t([[150000], [150001]]), s.t([3, 16]),
                                           scale=s.sc, return_lse=True)
    s.check("5 GiB", got)
