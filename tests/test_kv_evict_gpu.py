"""ssm_kv_mass_update and ssm_kv_evict on the GPU against the fp64 oracle, and a cache as a program
keeps it: filled, weighed, evicted, given back, grown again.

Bound of mass: an exponent is the score's (longctx_cases.spread: D) and lse's, log2(e) lse rounded twice, and
their difference rounded: D + 2 u (|s| + |lse|) in all, and 2^x within 2 u; a token's sum of n weights adds
(n / 16 + 8) u of itself (16 lanes of n / 16 each, joined, and added to what was there), all of it positive."""
import numpy as np
import pytest

from helpers import lib, report
from longctx_cases import EDGES, U, Paged, captured, n64
from oracle import longctx, paged

pytestmark = pytest.mark.gpu


class Step(Paged):
    """A step that took each request from `old` to `lens` tokens, q and lse of its rows, mass from before."""

    def __init__(self, device, seed, old, lens, H, Hk, d, cache, ps, layout="nhd", **kw):
        super().__init__(device, seed, lens, Hk, d, cache, ps, layout, **kw)
        import torch
        self.H, self.old = H, np.asarray(old)
        room = self.table.shape[1] * ps
        rows = np.maximum(np.minimum(self.lens, room) - np.maximum(self.old, 0), 0)
        self.starts = np.concatenate([[0], np.cumsum(rows)])
        self.pos = np.concatenate([np.arange(a, a + n) for a, n in zip(np.maximum(self.old, 0), rows)] + [np.zeros(0)]).astype(int)
        self.q = self.queries(int(rows.sum()), H, d)
        self.req = np.repeat(np.arange(len(rows)), rows)
        self.sc = d ** -0.5
        _, lse = paged.paged_attn_decode(n64(self.q), self.k64(), self.v64(), self.table[self.req], self.pos + 1, self.sc)
        self.lse = torch.tensor(lse, dtype=torch.float32, device=device)
        self.mass = torch.tensor(self.rng.random((self.pages, Hk, ps)), dtype=torch.float32, device=device)

    def call(self, mass=None):
        lib().ssm_kv_mass_update(self.q, self.k, self.lse, self.mass if mass is None else mass, self.t(self.table), self.t(self.starts),
                                 self.t(self.pos), self.t(self.old), self.t(self.lens), scale=self.sc, k_scale=self.scale)

    def check(self, name):
        was = n64(self.mass)
        k64, q64, lse = self.k64(), n64(self.q), n64(self.lse)
        want = longctx.mass_update(q64, k64, lse, was, self.table, self.starts, self.pos, self.old, self.lens, self.sc)
        self.call()
        got = n64(self.mass)
        touched = np.zeros(got.shape, bool)
        worst = 0.0
        for r in range(len(self.lens)):
            for j, p, i in longctx._tokens(self.table[r], self.lens[r], self.ps, self.pages):
                touched[p, :, i] = True
                rows = [t for t in range(self.starts[r], self.starts[r + 1]) if j <= self.pos[t]]
                n = len(rows) * self.H // self.Hk
                for g in range(self.Hk):
                    add = want[p, g, i] - (was[p, g, i] if j < self.old[r] else 0.0)
                    heads = range(g * (self.H // self.Hk), (g + 1) * (self.H // self.Hk))
                    x = np.abs(q64[rows][:, heads]) @ np.abs(k64[p, i, g]) * abs(self.sc) if rows else np.zeros(1)
                    low = np.abs(lse[rows][:, heads])
                    low = low[np.isfinite(low)].max(initial=0.0)
                    each = (self.d + 6) * U * x.max(initial=0.0) + 2 * U * (x.max(initial=0.0) + low) + 2 * U
                    tol = add * (1.5 * each + (n / 16 + 8) * U) + U * want[p, g, i] + 1e-37
                    worst = max(worst, abs(got[p, g, i] - want[p, g, i]) / tol)
        np.testing.assert_array_equal(got[~touched], was[~touched])
        report("mass " + name, of_bound=worst)
        assert worst <= 1.0, worst


GROWN = [min(max(0, n - 1 - 7 * (i % 3)), 300) for i, n in enumerate(EDGES)]
MASS = [  # old, lens, H, Hk, d, cache, page, layout
    ([0], [1], 1, 1, 64, "bf16", 16, "nhd"), (GROWN, EDGES, 4, 2, 64, "bf16", 16, "nhd"), (GROWN, EDGES, 4, 4, 128, "bf16", 1, "nhd"),
    (GROWN, EDGES, 6, 2, 128, "bf16", 8, "hnd"), (GROWN, EDGES, 5, 1, 80, "bf16", 24, "nhd"), (GROWN, EDGES, 17, 1, 96, "bf16", 7, "hnd"),
    (GROWN, EDGES, 2, 2, 192, "bf16", 64, "nhd"), (GROWN, EDGES, 4, 1, 256, "bf16", 16, "nhd"), (GROWN, EDGES, 3, 1, 8, "bf16", 5, "nhd"),
    (GROWN, EDGES, 8, 2, 128, "f8", 16, "nhd"), (GROWN, EDGES, 8, 1, 64, "f8", 64, "hnd"), (GROWN, EDGES, 4, 2, 192, "f8", 1, "nhd"),
    (GROWN, EDGES, 2, 1, 256, "f8", 8, "nhd"), (GROWN, EDGES, 6, 2, 16, "f8", 16, "nhd"), (GROWN, EDGES, 5, 1, 256, "f32", 24, "nhd"),
    (GROWN, EDGES, 4, 4, 128, "f32", 16, "hnd"), (GROWN, EDGES, 20, 1, 64, "f32", 8, "nhd"), (GROWN, EDGES, 3, 3, 192, "f32", 1, "nhd"),
    (GROWN, EDGES, 2, 1, 72, "f32", 16, "nhd"), ([0, 0, 40], [150, 333, 40], 4, 2, 64, "bf16", 16, "nhd"),
    ([0, 100], [97, 230], 3, 1, 128, "f8", 16, "nhd"), ([1000, 2999], [1001, 3000], 8, 2, 64, "bf16", 16, "nhd"),
    ([9] * 200, [10] * 200, 2, 2, 64, "f32", 16, "nhd"),
]


@pytest.mark.parametrize("case", MASS, ids=lambda c: "%d-%d-H%d-%d-d%d-%s-p%d-%s" % ((len(c[0]), max(c[1])) + c[2:]))
def test_mass_against_the_oracle(cuda_device, case):
    Step(cuda_device, 90 + case[4], *case).check(str(case[2:]))


def test_weights_of_a_step_add_up(cuda_device):
    """With the lse that the library's own attention gives, a request's weights add up to one a row and head."""
    import torch
    m = lib()
    s = Step(cuda_device, 91, [0, 50, 300], [700, 51, 400], 8, 2, 128, "bf16", 16, nan=False)
    o, s.lse = m.ssm_paged_attn_decode_fwd(s.q, s.k, s.v, s.t(s.table[s.req]), s.t(s.pos + 1), scale=s.sc, return_lse=True)
    s.mass.fill_(float("nan"))
    for r in range(3):
        j = np.arange(s.old[r])
        s.mass[torch.tensor(s.table[r, j // 16]), :, torch.tensor(j % 16)] = 0.0
    s.call()
    for r in range(3):
        j = np.arange(s.lens[r])
        got = n64(s.mass)[s.table[r, j // 16], :, j % 16].sum(0)
        rows = s.starts[r + 1] - s.starts[r]
        assert np.abs(got - rows * 4).max() <= rows * 4 * 1e-5


def test_rows_that_do_not_count(cuda_device):
    """A refused request's rows (places past its length), rows without a token (lse = -inf), places before 0, starts
    outside the rows, a request without rows; bad pages; NaN keys and NaN lse reach their own tokens and rows alone."""
    import torch
    s = Step(cuda_device, 92, [5, 30, 0, 8, 40], [9, 30, 20, 12, 44], 4, 2, 64, "f32", 16)
    # request 1 was refused: it keeps 30 tokens, and its 4 rows follow request 0's
    s.starts = np.array([0, 4, 8, 28, 32, 36])
    s.pos = np.concatenate([np.arange(5, 9), np.arange(30, 34), np.arange(20), np.arange(8, 12), np.arange(40, 44)])
    s.q = s.queries(36, 4, 64)
    s.lse = torch.tensor(s.rng.random((36, 4)) + 3.0, dtype=torch.float32, device=cuda_device)
    s.lse[10, 1], s.pos[9], s.pos[29] = -float("inf"), -1, -(1 << 31)
    s.table[4, 1] = s.pages
    s.check("rows that do not count")
    s.starts = np.array([-7, 4, 4, 2, 1 << 30, 1 << 30])      # cut to the rows, and never backwards
    was = n64(s.mass)
    s.call()
    got = n64(s.mass)
    fixed = [(0, 4), (4, 4), (4, 4), (2, 36), (36, 36)]
    want = was
    for r, (a, b) in enumerate(fixed):
        want = longctx.mass_update(n64(s.q)[a:b], s.k64(), n64(s.lse)[a:b], want, s.table[r:r + 1], [0, b - a], s.pos[a:b], s.old[r:r + 1],
                                   s.lens[r:r + 1], s.sc)
    np.testing.assert_allclose(got, want, rtol=1e-4, atol=1e-30)
    s = Step(cuda_device, 93, [0], [40], 2, 1, 64, "f32", 16, nan=False)
    s.k[s.table[0, 0], 7, 0, 3] = float("nan")
    s.call()
    assert n64(s.mass)[s.table[0, 0], 0, 7] != n64(s.mass)[s.table[0, 0], 0, 7]
    flat = n64(s.mass)[s.table[0, np.arange(40) // 16], 0, np.arange(40) % 16]
    assert np.isfinite(np.delete(flat, 7)).all()
    s.lse[20, 0] = float("nan")
    s.call()
    flat = n64(s.mass)[s.table[0, np.arange(40) // 16], 0, np.arange(40) % 16]
    assert np.isnan(flat[:21]).all() and np.isfinite(flat[21:]).all()


def test_no_rows_and_no_requests(cuda_device):
    """Without a row new tokens start at 0 and the others keep what they have; without a request nothing happens."""
    import torch
    s = Step(cuda_device, 94, [5, 3], [5, 3], 2, 1, 64, "f32", 16)
    s.old = np.array([3, 3])
    was = n64(s.mass)
    assert len(s.q) == 0
    s.call()
    got = n64(s.mass)
    assert (got[s.table[0, 0], 0, 3:5] == 0).all() and (got[s.table[0, 0], 0, :3] == was[s.table[0, 0], 0, :3]).all()
    got[s.table[0, 0], 0, 3:5] = was[s.table[0, 0], 0, 3:5]
    np.testing.assert_array_equal(got, was)
    i = lambda *n: torch.zeros(n, dtype=torch.int32, device=cuda_device)  # noqa: E731
    lib().ssm_kv_mass_update(s.q, s.k, s.lse, s.mass, i(0, 3), i(1), i(0), i(0), i(0), scale=1.0)
    n, kept = lib().ssm_kv_evict(s.k, s.v, s.mass, i(0, 3), i(0), budget=4)
    assert n.shape == (0,) and kept.shape == (0, 1, 4)


# -------------------------------------------------------------- eviction ----
def _bytes(t):
    import torch
    return t.contiguous().view(torch.uint8).cpu().numpy()


def _evict_and_check(c, mass, lens, budget, recent, **kw):
    import torch
    # values by their bytes: moved rows are the same bits, NaN too
    b = [_bytes(t).reshape(c.pages, c.ps, c.Hk, -1) for t in (c.k, c.v)]
    bits = mass.clone().view(torch.int32).cpu().numpy()
    _, _, _, length, kept = longctx.evict(b[0], b[1], n64(mass), c.table, lens, budget, recent)
    k, v, m, _, _ = longctx.evict(b[0], b[1], n64(mass), c.table, lens, budget, recent)
    got_n, got_kept = lib().ssm_kv_evict(c.k, c.v, mass, c.t(c.table), c.t(lens), budget=budget, recent=recent, **kw)
    np.testing.assert_array_equal(got_n.cpu().numpy(), length)
    np.testing.assert_array_equal(got_kept.cpu().numpy(), kept)
    np.testing.assert_array_equal(_bytes(c.k).reshape(k.shape), k)
    np.testing.assert_array_equal(_bytes(c.v).reshape(v.shape), v)
    np.testing.assert_array_equal(n64(mass), m)
    return bits


LONG = [1, 0, 17, 64, 65, 300, 1000, 777, -3]
EVICT = [  # lens, Hk, d, cache, page, layout, budget, recent
    (LONG, 2, 128, "bf16", 16, "nhd", 64, 8), (LONG, 1, 64, "bf16", 8, "hnd", 1, 0), (LONG, 1, 64, "bf16", 8, "hnd", 1, 1),
    (LONG, 3, 80, "bf16", 24, "nhd", 200, 0), (LONG, 2, 8, "bf16", 5, "nhd", 63, 63), (LONG, 1, 256, "bf16", 64, "hnd", 299, 100),
    (LONG, 4, 128, "f8", 16, "nhd", 100, 10), (LONG, 1, 16, "f8", 7, "nhd", 300, 299), (LONG, 2, 256, "f8", 64, "hnd", 999, 5),
    (LONG, 3, 72, "f32", 16, "nhd", 50, 20), (LONG, 2, 256, "f32", 1, "hnd", 256, 0), (LONG, 2, 64, "f32", 16, "nhd", 5000, 7),
    ([3000, 2999], 2, 128, "bf16", 16, "nhd", 2048, 100), ([9001], 1, 64, "bf16", 64, "hnd", 4000, 1), ([90] * 300, 2, 64, "f8", 16, "nhd", 64, 9),
    ([70000, 5], 1, 16, "f8", 64, "nhd", 66000, 100),
]


@pytest.mark.parametrize("case", EVICT, ids=lambda c: "%d-%d-Hk%d-d%d-%s-p%d-%s-b%d-%d" % ((len(c[0]), max(c[0])) + c[1:]))
def test_evict_against_the_oracle(cuda_device, case):
    import torch
    lens, Hk, d, cache, ps, layout, budget, recent = case
    c = Paged(cuda_device, 95 + d, lens, Hk, d, cache, ps, layout, nan=False)
    mass = torch.tensor(np.exp(2.5 * c.rng.standard_normal((c.pages, Hk, ps))), dtype=torch.float32, device=cuda_device)
    _evict_and_check(c, mass, lens, budget, recent)


def test_evict_among_equal_and_strange_mass(cuda_device):
    """Equal values (the earlier token stays), zeros of either sign, negative, infinite and NaN ones."""
    import torch
    rng = np.random.default_rng(5)
    for values in ([0.0], [1.0, 2.0], [0.0, -0.0], [-1.0, -2.0, 3.0], [float("inf"), -float("inf"), 1.0], [float("nan"), 2.0, float("inf")]):
        for budget, recent in ((100, 0), (333, 32), (901, 900)):
            c = Paged(cuda_device, 96, [1000, 2100, 902], 2, 16, "f32", 16, nan=False)
            mass = torch.tensor(rng.choice(values, (c.pages, 2, 16)), dtype=torch.float32, device=cuda_device)
            _evict_and_check(c, mass, c.lens, budget, recent)


def test_evict_moves_a_little_and_a_lot(cuda_device):
    """The first token goes (all move by one), the last that may (one moves), every second one, and none before the last."""
    import torch
    for gone in ([0], [1999 - 33], list(range(0, 1900, 2)), [0, 1, 2], list(range(1000, 1900))):
        c = Paged(cuda_device, 97, [2000], 2, 128, "bf16", 16, nan=False)
        mass = torch.ones((c.pages, 2, 16), device=cuda_device)
        for j in gone:
            mass[c.table[0, j // 16], :, j % 16] = 0.5
        _evict_and_check(c, mass, [2000], 2000 - len(gone), 32)


def test_evict_bad_pages_long_lengths_and_given_tensors(cuda_device):
    import torch
    c = Paged(cuda_device, 98, [500, 400, 300], 2, 64, "bf16", 16, nan=False)
    c.table[0, 3], c.table[0, 20], c.table[1, 24], c.table[2, 18] = -1, c.pages, 1 << 30, -(1 << 31)
    mass = torch.tensor(c.rng.random((c.pages, 2, 16)), dtype=torch.float32, device=cuda_device)
    n, kept = torch.empty(3, dtype=torch.int32, device=cuda_device), torch.empty((3, 2, 250), dtype=torch.int32, device=cuda_device)
    _evict_and_check(c, mass, [1 << 30, 400, 300], 250, 50, len_out=n, kept=kept)
    assert n.tolist() == [250] * 3 and (kept >= 0).all()
    # and where the kept ones do not all have a page to go to or to come from
    c = Paged(cuda_device, 99, [64], 1, 16, "f32", 4, nan=False)
    c.table[0, ::2] = -1
    _evict_and_check(c, torch.tensor(c.rng.random((c.pages, 1, 4)), dtype=torch.float32, device=cuda_device), [64], 40, 3)


def test_evict_in_a_graph_and_on_another_stream(cuda_device):
    import torch
    m = lib()
    c = Paged(cuda_device, 100, [600, 20, 333, 1], 2, 128, "bf16", 16, nan=False)
    table, lens = c.t(c.table), c.t([600, 20, 333, 1])
    mass = torch.rand((c.pages, 2, 16), device=cuda_device)
    n, kept = torch.empty(4, dtype=torch.int32, device=cuda_device), torch.empty((4, 2, 64), dtype=torch.int32, device=cuda_device)
    call = lambda: m.ssm_kv_evict(c.k, c.v, mass, table, lens, budget=64, recent=10, len_out=n, kept=kept)  # noqa: E731
    g = captured(call)
    side = torch.cuda.Stream()
    for new in ([600, 20, 333, 1], [64, 65, 0, 16], [608, 32, 336, 5]):
        lens.copy_(torch.tensor(new))
        mass.copy_(torch.rand_like(mass))
        c.k.copy_(torch.randn_like(c.k))
        state = [t.clone() for t in (c.k, c.v, mass)]
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (c.k, c.v, mass, n, kept)]
        for t, s in zip((c.k, c.v, mass), state):
            t.copy_(s)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (c.k, c.v, mass, n, kept)))
        want = longctx.evict(np.zeros((c.pages, 16, 2, 1)), np.zeros((c.pages, 16, 2, 1)), n64(state[2]), c.table, new, 64, 10)
        np.testing.assert_array_equal(kept.cpu().numpy(), want[4])


# --------------------------------------------------------- all of them ----
@pytest.mark.parametrize("cache", ["bf16", "f8", "f32"])
def test_a_cache_as_a_program_keeps_it(cuda_device, cache):
    """Requests behind a shared prefix: pages taken, keys written, attention with the prefix, weights gathered, tokens
    evicted once there are too many, pages given back, bounds kept up, and attention over chosen pages; every step against
    the oracle on the cache as it stands, and the free pages counted."""
    import torch
    from longctx_cases import TYPES, compare, i32
    m = lib()
    dev, rng = cuda_device, np.random.default_rng(101)
    B, H, Hk, d, ps, P, cols, budget = 3, 4, 2, 64, 8, 60, 16, 48
    dt = torch.float32 if cache == "f32" else torch.bfloat16
    scale = 0.03125 if cache == "f8" else 1.0
    kc, vc = (torch.zeros((P, ps, Hk, d), device=dev).to(TYPES[cache]) for _ in range(2))
    table, ring, head = i32(np.zeros((B + 1, cols)), dev), i32(rng.permutation(P), dev), i32([0, P], dev)
    mass = torch.full((P, Hk, ps), float("nan"), device=dev)
    bounds = torch.zeros((P, Hk, 2, d), device=dev).to(TYPES[cache])
    none = torch.ones(d, device=dev)
    freq = torch.rand(8, device=dev)
    held = i32([0] * (B + 1), dev)
    # row B is the prefix: its tokens come first and are never evicted
    for step, grow in enumerate(([40, 0, 7, 90], [1, 60, 1, 0], [30, 1, 1, 0], [1, 1, 45, 0], [1, 1, 1, 0])):
        old = held
        want = (held + i32(grow, dev)).int()
        T = sum(grow)
        s = m.ssm_kv_pages_step(old, want, table, ring, head, page_size=ps, n_tokens=T)
        held, head = s["len"], s["ring"]
        assert int(s["denied"]) == 0
        q, k, v = (torch.tensor(rng.standard_normal((T, h, d)), device=dev).to(dt) for h in (H, Hk, Hk))
        q = m.ssm_qk_norm_rope_cache_fwd(q, k, v, none, none, freq, s["positions"], s["slots"], kc, vc, k_scale=scale, v_scale=scale)
        n = held.cpu().numpy()
        tab = table.cpu().numpy()
        k64, v64 = n64(kc) * scale, n64(vc) * scale
        # attention of the step's rows over their own tokens, and what those gathered
        req = s["request"].long()
        _, lse = m.ssm_paged_attn_decode_fwd(q, kc, vc, table[req].contiguous(), s["positions"] + 1, scale=0.1, k_scale=scale, v_scale=scale,
                                             return_lse=True)
        before = n64(mass)
        m.ssm_kv_mass_update(q, kc, lse, mass, table, s["starts"], s["positions"], old, held, scale=0.1, k_scale=scale)
        want_mass = longctx.mass_update(n64(q), k64, n64(lse), before, tab, s["starts"].cpu().numpy(), s["positions"].cpu().numpy(),
                                        old.cpu().numpy(), n, 0.1)
        np.testing.assert_allclose(n64(mass), want_mass, rtol=2e-5, atol=1e-30)
        m.ssm_kv_page_bounds_update(kc, bounds, table, old, held)
        # the newest row of each request, with the prefix
        last = (s["starts"][1:B + 1] - 1).long().clamp(min=0)
        ql = q[last].contiguous()
        got = m.ssm_prefix_attn_decode_fwd(ql, kc, vc, i32([0] * B, dev), table[B:], held[B:].contiguous(), table[:B], held[:B].contiguous(),
                                           scale=0.1, k_scale=scale, v_scale=scale, return_lse=True)
        want_o = longctx.prefix_attn_decode(n64(ql), k64, v64, [0] * B, tab[B:], n[B:], tab[:B], n[:B], 0.1)

        def rows_of(r, h):
            t = longctx._tokens(tab[B], n[B], ps, P) + longctx._tokens(tab[r], n[r], ps, P)
            return k64[[x[1] for x in t], [x[2] for x in t], h * Hk // H], v64[[x[1] for x in t], [x[2] for x in t], h * Hk // H]
        worst = compare(got, want_o, rows_of, ql, 0.1, cache != "f32", 2.0 ** -17 if cache != "f32" else 0.0)
        assert max(worst) <= 1.0, worst
        # over chosen pages: the bounds hold every key that is there
        sel = m.ssm_kv_page_select_fwd(ql, bounds, table[:B], held[:B].contiguous(), page_size=ps, top_k=4, first=1, last=1)
        np.testing.assert_array_equal(sel.cpu().numpy(), longctx.page_select(n64(ql), n64(bounds), tab[:B], n[:B], ps, 4, 1, 1))
        got = m.ssm_select_attn_decode_fwd(ql, kc, vc, table[:B], held[:B].contiguous(), sel, scale=0.1, k_scale=scale, v_scale=scale,
                                           return_lse=True)
        want_o = longctx.select_attn_decode(n64(ql), k64, v64, tab[:B], n[:B], sel.cpu().numpy(), 0.1)

        def chosen(r, h):
            g = h * Hk // H
            keep = set(sel[r, g].tolist())
            t = [x for x in longctx._tokens(tab[r], n[r], ps, P) if x[0] // ps in keep]
            return k64[[x[1] for x in t], [x[2] for x in t], g], v64[[x[1] for x in t], [x[2] for x in t], g]
        worst = compare(got, want_o, chosen, ql, 0.1, cache != "f32", 0.0)
        assert max(worst) <= 1.0, worst
        # too many tokens: the least weighty go, their pages come back, and what moved has bounds anew
        full = held.clone()
        full[B] = 0                              # (the prefix has a length of its own: left out here)
        state = [_bytes(x).reshape(P, ps, Hk, -1) for x in (kc, vc)] + [n64(mass)]
        cut, kept = m.ssm_kv_evict(kc, vc, mass, table, full, budget=budget, recent=8)
        wk, wv, wm, wn, wkept = longctx.evict(*state, tab, full.cpu().numpy(), budget, 8)
        np.testing.assert_array_equal(kept.cpu().numpy(), wkept)
        np.testing.assert_array_equal(_bytes(kc).reshape(wk.shape), wk)
        np.testing.assert_array_equal(_bytes(vc).reshape(wv.shape), wv)
        np.testing.assert_array_equal(n64(mass), wm)
        cut = torch.cat([cut[:B], held[B:]])
        free = int(head[1])
        s = m.ssm_kv_pages_step(held, cut, table, ring, head, page_size=ps, n_tokens=0)
        pages = lambda x: -(-x.cpu().numpy() // ps)  # noqa: E731
        assert int(s["ring"][1]) == free + (pages(held) - pages(cut)).sum()
        moved = torch.where(cut < held, 0, cut).int()
        held, head = s["len"], s["ring"]
        m.ssm_kv_page_bounds_update(kc, bounds, table, moved, held)
        assert (held[:B] <= budget).all()
