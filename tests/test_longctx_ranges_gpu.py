"""The long-context operators where their ranges are wide: many rows behind tables with room for long prefixes,
caches past 4 GiB, prompts whose rows come in any order, long budgets in a graph, and calls on two streams at once.
Bounds are those of the operators' own tests; what is compared between two calls is equal bit for bit."""
import numpy as np
import pytest

from helpers import lib
from longctx_cases import EDGES, TYPES, Paged, captured, n64
from test_kv_evict_gpu import Step
from test_prefix_attn_gpu import Shared

pytestmark = pytest.mark.gpu

# prefix lengths, prefix of each row, own lengths, H, Hk, d, cache, page, layout; room for 60000 tokens of a prefix
ROOM = 60000
MANY = [
    ([300], [0] * 80, [i % 9 for i in range(80)], 8, 2, 128, "bf16", 16, "nhd"),
    ([700, 33, 0, 257], [0] * 37 + [1] * 13 + [-1, 9] + [2] * 13 + [3] * 35, EDGES * 5, 12, 2, 64, "bf16", 8, "hnd"),
    ([100, 200, 300], [i % 3 for i in range(200)], EDGES * 10, 3, 1, 80, "bf16", 24, "nhd"),
    ([129], [0] * 5, [0, 1, 2, 3, 4], 140, 1, 96, "bf16", 16, "nhd"),                         # more heads than a block's columns
    ([600], [0] * 80, EDGES * 4, 8, 2, 128, "f8", 16, "nhd"),
    ([1000, 100], [0] * 50 + [1] * 50, EDGES * 5, 8, 1, 64, "f8", 64, "hnd"),
    ([129], [0] * 100, EDGES * 5, 6, 1, 16, "f8", 7, "nhd"),
    ([200, 70], [0] * 62 + [1] * 78, EDGES * 7, 4, 1, 128, "f32", 16, "hnd"),
    ([333], [0] * 60, EDGES * 3, 20, 2, 72, "f32", 24, "nhd"),
    ([150], [0] * 160, EDGES * 8, 4, 4, 64, "f32", 8, "nhd"),
    ([385], [0] * 40, EDGES * 2, 16, 1, 256, "bf16", 16, "nhd"),
    ([385], [0] * 40, EDGES * 2, 16, 1, 192, "f8", 16, "hnd"),
]


def _wide(s):
    s.ptable = np.pad(s.ptable, ((0, 0), (0, -(-ROOM // s.ps) - s.ptable.shape[1])), constant_values=-1)
    return s


@pytest.mark.parametrize("case", MANY, ids=lambda c: "%d-%d-%d-H%d-%d-d%d-%s-p%d-%s" % ((max(c[0]), len(c[0]), len(c[2])) + c[3:]))
def test_many_rows_with_room_for_long_prefixes(cuda_device, case):
    _wide(Shared(cuda_device, 110 + case[5], *case)).check("room " + str(case[3:]))


def test_infinite_and_nan_keys_of_many_rows(cuda_device):
    """-inf scores weigh nothing and a prefix of only those is empty; a NaN key reaches the rows of its prefix alone; rows of
    zeros in a cache that is all NaN elsewhere."""
    for cache in ("f32", "bf16"):
        s = _wide(Shared(cuda_device, 120, [80, 80, 80], [0] * 50 + [1] * 50 + [2] * 50, [0, 3] * 75, 4, 1, 64, cache, 16))
        s.q = s.q.abs() + 0.1
        at = lambda p, j: (int(s.ptable[p, j // 16]), j % 16)  # noqa: E731
        for j in range(3, 40):
            s.k[at(0, j)][0, 5] = -float("inf")
        for j in range(80):
            s.k[at(1, j)][0, 7] = -float("inf")
        s.k[at(2, 11)][0, 0] = float("nan")
        o, lse = s.call()
        o, lse = n64(o), n64(lse)
        assert np.isfinite(o[:100]).all() and np.isnan(o[100:]).all() and np.isnan(lse[100:]).all()
        assert (o[50:100:2] == 0).all() and np.isneginf(lse[50:100:2]).all() and np.isfinite(lse[:50]).all()


def test_bad_pages_and_long_lengths_of_many_rows(cuda_device):
    """Pages outside the cache hold no token, lengths end with their table, tables and q are strided, and the workspace holds
    NaN before."""
    import torch
    m = lib()
    for cache, d in (("bf16", 128), ("f8", 64), ("f32", 64)):
        s = _wide(Shared(cuda_device, 122, [200, 90], [i % 2 for i in range(90)], [i % 70 for i in range(90)], 8, 2, d, cache, 16))
        s.ptable[0, 3], s.ptable[0, 5], s.ptable[1, 0], s.own[1, 0] = -1, s.pages, 1 << 30, -7
        s.ptable[0, 12] = -(1 << 31)
        s.plens = np.array([1 << 30, 90])                     # every place of the table, most of them without a page
        s.rows = s.rows.copy()
        s.rows[5], s.rows[6] = -1, 1 << 30
        s.k, s.v = (torch.nan_to_num(c.float(), nan=0.5).to(c.dtype) for c in (s.k, s.v))
        proj = torch.randn((90, 8 * d + 64), device=cuda_device).to(s.q.dtype)
        s.q = proj[:, 64:].unflatten(1, (8, d))
        big = torch.full((90, s.own.shape[1] + 4), -1, dtype=torch.int32, device=cuda_device)
        big[:, :s.own.shape[1]] = s.t(s.own)
        pbig = torch.full((2, s.ptable.shape[1] + 3), 5, dtype=torch.int32, device=cuda_device)
        pbig[:, :s.ptable.shape[1]] = s.t(s.ptable)
        ws = torch.full((m.ssm_prefix_attn_decode_fwd_workspace_size(90, 8, 2, d, s.ptable.shape[1], s.own.shape[1], 16),), 255,
                        dtype=torch.uint8, device=cuda_device)
        got = m.ssm_prefix_attn_decode_fwd(s.q, s.k, s.v, s.t(s.prefix), pbig[:, :s.ptable.shape[1]], s.t(s.plens), big[:, :s.own.shape[1]],
                                           s.t(s.rows), scale=s.sc, k_scale=s.scale, v_scale=s.scale, return_lse=True, workspace=ws)
        s.check("bad pages of many rows " + cache, got)


def test_many_rows_in_a_graph(cuda_device):
    """Captured once, two graphs with one workspace; everything changes in place between replays, with eager calls between."""
    import torch
    m = lib()
    for d, cache in ((128, "bf16"), (64, "f8"), (128, "f32")):
        s = _wide(Shared(cuda_device, 121, [600, 300], [i % 2 for i in range(90)], [i % 60 for i in range(90)], 8, 2, d, cache, 16, nan=False))
        prefix, plens, rows, own, pt = s.t(s.prefix), s.t(s.plens), s.t(s.rows), s.t(np.maximum(s.own, 0)), s.t(np.maximum(s.ptable, 0))
        o, lse = torch.empty_like(s.q), torch.empty((90, 8), device=cuda_device)
        ws = torch.empty(m.ssm_prefix_attn_decode_fwd_workspace_size(90, 8, 2, d, pt.shape[1], own.shape[1], 16), dtype=torch.uint8,
                         device=cuda_device)

        def call(scale=0.09):
            m.ssm_prefix_attn_decode_fwd(s.q, s.k, s.v, prefix, pt, plens, own, rows, scale=scale, k_scale=s.scale, v_scale=s.scale, o=o,
                                         lse=lse, workspace=ws)
        graphs = [(captured(lambda x=x: call(x)), x) for x in (0.09, 0.2)]
        rng = np.random.default_rng(5)
        for pl in ([600, 300], [17, 608], [0, 0]):
            prefix.copy_(torch.tensor(rng.integers(-1, 3, 90)))
            plens.copy_(torch.tensor(pl))
            rows.copy_(torch.tensor(rng.integers(0, 60, 90)))
            s.q.copy_(torch.randn_like(s.q))
            for g, x in graphs:
                o.fill_(7.0)
                g.replay()
                torch.cuda.synchronize()
                a, b = o.clone(), lse.clone()
                o.fill_(9.0)
                call(x)
                torch.cuda.synchronize()
                assert torch.equal(a, o) and torch.equal(b, lse)


def _far(c, pages, ids):
    """c's caches with its page i at ids[i] of `pages`, and its table."""
    import torch
    out = []
    for t in (c.k, c.v):
        big = torch.zeros((pages, c.ps, c.Hk, c.d), dtype=t.dtype, device=c.device)
        big[torch.tensor(ids, device=c.device)] = t.contiguous()
        out.append(big)
    return out, np.where(c.table >= 0, np.asarray(ids)[np.maximum(c.table, 0)], -1)


@pytest.mark.parametrize("ps", [16, 1])
def test_caches_past_4_gib(cuda_device, ps):
    """Pages anywhere in caches of 5 GiB a tensor: bounds, choice, attention over it, gathered weight and eviction give what they
    give in a small cache.  With pages of one token the bounds are 10 GiB too."""
    import torch
    m = lib()
    P, H, Hk, d = 163840 * 16 // ps, 16, 8, 128
    s = Step(cuda_device, 130, [0, 60, 20], [50, 61, 64], H, Hk, d, "bf16", ps, nan=False)
    ids = np.concatenate([[P - 1, P - 2, 0], 3 + s.rng.permutation(P - 6)[:s.pages - 3]])
    (k, v), table = _far(s, P, ids)
    at, tab, small = torch.tensor(ids, device=cuda_device), s.t(table), s.t(s.table)
    old, lens = s.t(s.old), s.t(s.lens)
    bounds = [torch.zeros((n, Hk, 2, d), dtype=torch.bfloat16, device=cuda_device) for n in (s.pages, P)]
    m.ssm_kv_page_bounds_update(s.k, bounds[0], small, s.t([0, 0, 0]), lens)
    m.ssm_kv_page_bounds_update(k, bounds[1], tab, s.t([0, 0, 0]), lens)
    assert torch.equal(bounds[0], bounds[1][at])
    q = s.queries(3, H, d)
    sel = [m.ssm_kv_page_select_fwd(q, b, t, lens, page_size=ps, top_k=2 * 16 // ps, first=1, last=1) for b, t in zip(bounds, (small, tab))]
    assert torch.equal(sel[0], sel[1])
    del bounds
    got = [m.ssm_select_attn_decode_fwd(q, kk, vv, t, lens, sel[0], scale=0.1, return_lse=True) for kk, vv, t in ((s.k, s.v, small), (k, v, tab))]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    mass = torch.zeros((P, Hk, ps), device=cuda_device)
    mass[at] = s.mass
    s.call()
    m.ssm_kv_mass_update(s.q, k, s.lse, mass, tab, s.t(s.starts), s.t(s.pos), old, lens, scale=s.sc)
    assert torch.equal(mass[at], s.mass)
    # one row a request as well
    one, last = s.t([0, 1, 2, 3]), (s.lens - 1)
    rows = torch.tensor(s.starts[1:] - 1, device=cuda_device)
    for kk, mm, t in ((s.k, s.mass, small), (k, mass, tab)):
        m.ssm_kv_mass_update(s.q[rows].contiguous(), kk, s.lse[rows].contiguous(), mm, t, one, s.t(last), lens, lens, scale=s.sc)
    assert torch.equal(mass[at], s.mass)
    kept = [m.ssm_kv_evict(kk, vv, mm, t, lens, budget=37, recent=5) for kk, vv, mm, t in ((s.k, s.v, s.mass, small), (k, v, mass, tab))]
    assert torch.equal(kept[0][0], kept[1][0]) and torch.equal(kept[0][1], kept[1][1])
    assert torch.equal(k[at], s.k) and torch.equal(v[at], s.v) and torch.equal(mass[at], s.mass)


@pytest.mark.parametrize("cache", ["bf16", "f8", "f32"])
def test_gathered_weight_of_rows_in_any_order(cuda_device, cache):
    """A prompt's rows shuffled, some at one place twice, and a request whose rows all look back less than its tokens."""
    import torch
    s = Step(cuda_device, 131, [0, 100, 5], [333, 390, 300], 6, 2, 64, cache, 16)
    for a, b in zip(s.starts, s.starts[1:]):
        order = a + s.rng.permutation(b - a)
        order[:7] = order[7:14]
        s.pos[a:b], s.q[a:b], s.lse[a:b] = s.pos[order], s.q[torch.tensor(order)], s.lse[torch.tensor(order)]
    s.check("any order " + cache)
    s.pos = np.minimum(s.pos, 40)
    s.lse = s.lse + 4.0
    s.check("places before 41 " + cache)


def test_a_long_budget_in_a_graph(cuda_device):
    """A budget of more tokens than one pass of a request's blocks moves."""
    import torch
    m = lib()
    c = Paged(cuda_device, 132, [40000, 34000], 1, 16, "bf16", 64, nan=False)
    table, lens, mass = c.t(c.table), c.t([40000, 34000]), torch.rand((c.pages, 1, 64), device=cuda_device)
    n, kept = torch.empty(2, dtype=torch.int32, device=cuda_device), torch.empty((2, 1, 33000), dtype=torch.int32, device=cuda_device)
    call = lambda: m.ssm_kv_evict(c.k, c.v, mass, table, lens, budget=33000, recent=10, len_out=n, kept=kept)  # noqa: E731
    g = captured(call)
    for new in ([40000, 34000], [33001, 5], [39999, 33000]):
        lens.copy_(torch.tensor(new))
        mass.copy_(torch.rand_like(mass))
        c.k.copy_(torch.randn_like(c.k))
        state = [t.clone() for t in (c.k, c.v, mass)]
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (c.k, c.v, mass, n, kept)]
        for t, s in zip((c.k, c.v, mass), state):
            t.copy_(s)
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (c.k, c.v, mass, n, kept)))


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_two_streams_at_once(cuda_device, cache):
    """Two requests' batches on two streams, call by call, each with workspaces of its own: what each gives alone."""
    import torch
    m = lib()
    work = [_wide(Shared(cuda_device, 140 + i, [500, 100], [i % 2 for i in range(60)], EDGES * 3, 8, 2, 64, cache, 16)) for i in range(2)]
    steps = [Step(cuda_device, 142 + i, [0, 100, 5], [233, 290, 200], 4, 2, 64, cache, 16, nan=False) for i in range(2)]
    bounds = [torch.randn((s.pages, 2, 2, 64), device=cuda_device).to(TYPES[cache]) for s in steps]

    def run(i):
        s, t = work[i], steps[i]
        mass, k, v = t.mass.clone(), t.k.clone(), t.v.clone()
        out = list(s.call())
        t.call(mass)
        q, lens, table = t.q[:3], t.t(t.lens), t.t(t.table)
        sel = m.ssm_kv_page_select_fwd(q, bounds[i], table, lens, page_size=16, top_k=5)
        out += [sel, *m.ssm_select_attn_decode_fwd(q, t.k, t.v, table, lens, sel, scale=0.1, return_lse=True)]
        out += [*m.ssm_kv_evict(k, v, mass, table, lens, budget=150, recent=20), k, v, mass]
        return out

    alone = [run(0), run(1)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        both = []
        for i, side in enumerate(sides):
            with torch.cuda.stream(side):
                both.append(run(i))
        for side in sides:
            side.synchronize()
        for a, b in zip(alone, both):
            for x, y in zip(a, b):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
