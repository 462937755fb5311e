"""ssm_kv_page_bounds_update, ssm_kv_page_select_fwd and ssm_select_attn_decode_fwd on the GPU
against the fp64 oracle.  Bounds and choices are exact; attention is within the bound of
longctx_cases.attention_bound (three bf16 values in place of a weight keep all of its bits)."""
import numpy as np
import pytest

from helpers import lib, report
from longctx_cases import EDGES, TYPES, Paged, captured, compare, n64
from oracle import longctx

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- bounds ----
BOUNDS = [  # lens, Hk, d, cache, page, layout
    (EDGES, 2, 128, "bf16", 16, "nhd"), (EDGES, 1, 64, "bf16", 8, "hnd"), (EDGES, 3, 80, "bf16", 24, "nhd"),
    (EDGES, 2, 8, "bf16", 5, "nhd"), (EDGES, 1, 256, "bf16", 64, "hnd"), (EDGES, 4, 128, "f8", 16, "nhd"),
    (EDGES, 1, 16, "f8", 7, "nhd"), (EDGES, 2, 256, "f8", 64, "hnd"), (EDGES, 3, 72, "f32", 16, "nhd"),
    (EDGES, 2, 256, "f32", 1, "hnd"), ([3000, 0, 1], 8, 192, "f8", 128, "nhd"), ([1] * 700, 2, 64, "bf16", 16, "nhd"),
    ([7] * 4096, 1, 16, "bf16", 4, "nhd"),
]


def _bounds(c, had):
    import torch
    t = torch.tensor(had, dtype=torch.float32).to(TYPES[c.cache]).to(c.device)
    return t.contiguous()


@pytest.mark.parametrize("case", BOUNDS, ids=lambda c: "%d-%d-Hk%d-d%d-%s-p%d-%s" % ((len(c[0]), max(c[0])) + c[1:]))
def test_bounds_in_steps(cuda_device, case):
    """From nothing, then grown in two uneven steps: each page's smallest and largest keys, and other pages' bounds as
    they were."""
    m, (lens, Hk, d, cache, ps, layout) = lib(), case
    c = Paged(cuda_device, 60 + d, lens, Hk, d, cache, ps, layout)
    b = _bounds(c, np.full((c.pages, Hk, 2, d), 3.0))
    want = n64(b)
    k = n64(c.k)
    top = np.maximum(c.lens, 0)
    steps = [np.zeros_like(top), top // 3, top // 3 + (top > 2), top]
    for old, new in zip(steps, steps[1:]):
        m.ssm_kv_page_bounds_update(c.k, b, c.t(c.table), c.t(old), c.t(new))
        want = longctx.page_bounds(k, want, c.table, old, new)
        np.testing.assert_array_equal(n64(b), want)
    # nothing new, shrunk, negative: as they were
    for old, new in ((top, top), (top, top // 2), (top + 5, -top)):
        m.ssm_kv_page_bounds_update(c.k, b, c.t(c.table), c.t(old), c.t(new))
    np.testing.assert_array_equal(n64(b), want)


def test_bounds_of_nan_infinite_and_bad_pages(cuda_device):
    import torch
    m = lib()
    for cache in ("bf16", "f32", "f8"):
        c = Paged(cuda_device, 61, [40, 33, 20], 2, 64, cache, 16)
        f = c.k.float()
        f[c.table[0, 0], 3, 1, 5] = float("nan")
        f[c.table[0, 1], 2, 0, 6] = -0.0
        if cache != "f8":
            f[c.table[1, 0], 0, 0, 7], f[c.table[1, 1], 9, 1, 8] = float("inf"), -float("inf")
        c.k = f.to(TYPES[cache])
        table = c.table.copy()
        table[2, 0], table[2, 1] = -1, c.pages
        b = _bounds(c, np.full((c.pages, 2, 2, 64), 3.0))
        want = longctx.page_bounds(n64(c.k), n64(b), table, [0, 0, 0], [40, 33, 1 << 30])
        m.ssm_kv_page_bounds_update(c.k, b, c.t(table), c.t([0, 0, -5]), c.t([40, 33, 1 << 30]))
        np.testing.assert_array_equal(n64(b), want)
        assert torch.isnan(b[c.table[0, 0], 1, :, 5].float()).all()
        # a NaN that a page had stays
        c2 = Paged(cuda_device, 62, [40], 2, 64, cache, 16)
        b = _bounds(c2, np.full((c2.pages, 2, 2, 64), float("nan")))
        m.ssm_kv_page_bounds_update(c2.k, b, c2.t(c2.table), c2.t([20]), c2.t([40]))
        assert torch.isnan(b[c2.table[0, 1]].float()).all() and torch.isfinite(b[c2.table[0, 2]].float()).all()


def test_bounds_no_requests(cuda_device):
    import torch
    k, i = torch.zeros((2, 16, 1, 64), device=cuda_device), lambda *n: torch.zeros(n, dtype=torch.int32, device=cuda_device)
    b = torch.full((2, 1, 2, 64), 5.0, device=cuda_device)
    lib().ssm_kv_page_bounds_update(k, b, i(0, 3), i(0), i(0))
    assert (b == 5).all()


# ---------------------------------------------------------------- choice ----
def _random_bounds(c, rng):
    b = np.sort(rng.standard_normal((c.pages, c.Hk, 2, c.d)), axis=2) / c.scale
    return _bounds(c, b)


def _select(c, q, b, lens, top_k, first, last, **kw):
    return lib().ssm_kv_page_select_fwd(q, b, c.t(c.table), c.t(lens), page_size=c.ps, top_k=top_k, first=first, last=last, **kw)


LONG = [1, 0, 17, 64, 65, 300, 1000, 2500, -3]
SELECT = [  # lens, H, Hk, d, cache, page, top_k, first, last
    (LONG, 8, 2, 128, "bf16", 16, 20, 1, 4), (LONG, 4, 4, 64, "bf16", 8, 1, 0, 0), (LONG, 5, 1, 80, "bf16", 24, 7, 0, 1),
    (LONG, 40, 2, 72, "bf16", 16, 33, 2, 0), (LONG, 3, 1, 8, "bf16", 5, 40, 0, 3), (LONG, 2, 2, 256, "bf16", 64, 4, 1, 1),
    (LONG, 17, 1, 192, "bf16", 16, 16, 0, 0), (LONG, 8, 2, 128, "f8", 16, 50, 0, 1), (LONG, 6, 2, 16, "f8", 16, 9, 3, 3),
    (LONG, 5, 1, 256, "f8", 8, 100, 10, 20), (LONG, 6, 3, 72, "f32", 16, 17, 0, 1), (LONG, 9, 1, 256, "f32", 1, 200, 5, 7),
    (LONG, 2, 1, 64, "f32", 16, 10, 5, 5), (LONG, 4, 2, 64, "bf16", 16, 1000, 1, 1), ([9000, 8193, 20000], 2, 1, 16, "bf16", 1, 300, 2, 9),
    ([700] * 300, 2, 2, 64, "bf16", 16, 12, 1, 1),
]


@pytest.mark.parametrize("case", SELECT, ids=lambda c: "%d-%d-H%d-%d-d%d-%s-p%d-k%d-%d-%d" % ((len(c[0]), max(c[0])) + c[1:]))
def test_choice_against_the_oracle(cuda_device, case):
    lens, H, Hk, d, cache, ps, top_k, first, last = case
    c = Paged(cuda_device, 70 + d, lens, Hk, d, cache, ps, nan=False)
    q, b = c.queries(len(lens), H, d), _random_bounds(c, c.rng)
    got = _select(c, q, b, lens, top_k, first, last)
    want = longctx.page_select(n64(q), n64(b), c.table, lens, ps, top_k, first, last)
    np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_choice_among_equal_scores(cuda_device):
    """Scores of a few whole values, so that most pages are equal and the lowest are to be taken; all of them zero, of
    either sign; and infinite and NaN ones, which come in order."""
    import torch
    c = Paged(cuda_device, 71, [3000, 2000, 4100], 2, 16, "f32", 4, nan=False)
    rng = np.random.default_rng(3)
    q = torch.ones((3, 2, 16), device=cuda_device)
    for values in ([0, 1, 2], [0, -0.0], [5], [-3, -3, -3, 4], [float("inf"), -float("inf"), 1, 2], [float("nan"), 3, float("inf")]):
        b = np.zeros((c.pages, 2, 2, 16))
        b[..., 1, 3] = rng.choice(values, (c.pages, 2))
        b = _bounds(c, b)
        for k, first, last in ((1, 0, 0), (100, 0, 0), (101, 3, 7), (700, 1, 1)):
            got = _select(c, q, b, c.lens, k, first, last)
            want = longctx.page_select(n64(q), n64(b), c.table, c.lens, 4, k, first, last)
            np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=str((values, k, first, last)))


def test_scores_that_lie_close_together(cuda_device):
    """Pages whose scores differ in the last of 24 bits, with terms of both signs that are 2^20 times larger: the order is
    that of the 64-bit sums."""
    import torch
    c = Paged(cuda_device, 72, [1600], 1, 64, "f32", 16, nan=False)
    rng = np.random.default_rng(4)
    q = torch.ones((1, 1, 64), device=cuda_device)
    b = np.zeros((c.pages, 1, 2, 64))
    big = rng.integers(1, 9, (c.pages, 31)) * 2.0 ** 20
    b[:, 0, 1, :31], b[:, 0, 1, 31:62] = big, -big[:, ::-1]
    b[:, 0, 1, 62] = 1.0
    b[:, 0, 1, 63] = rng.permutation(c.pages) * 2.0 ** -23
    b = _bounds(c, b)
    for k in (1, 13, 50, 99):
        got = _select(c, q, b, [1600], k, 0, 0)
        np.testing.assert_array_equal(got.cpu().numpy(), longctx.page_select(n64(q), n64(b), c.table, [1600], 16, k, 0, 0))


def test_choice_bad_pages_strides_and_given_tensors(cuda_device):
    import torch
    m = lib()
    c = Paged(cuda_device, 73, [1000, 900, 90], 2, 64, "bf16", 16, nan=False)
    c.table[0, 5], c.table[0, 6], c.table[1, :40] = -1, c.pages, 1 << 30
    cols = c.table.shape[1]
    big = torch.zeros((3, cols + 5), dtype=torch.int32, device=cuda_device)
    big[:, :cols] = c.t(c.table)
    q = torch.randn((3, 1024), device=cuda_device).to(torch.bfloat16)[:, 64:320].view(3, 4, 64)
    b = _random_bounds(c, c.rng)
    ws = torch.full((m.ssm_kv_page_select_fwd_workspace_size(3, 2, cols, 30),), 255, dtype=torch.uint8, device=cuda_device)
    out = torch.full((3, 2, 30), 77, dtype=torch.int32, device=cuda_device)
    lens = [1 << 30, 900, 90]
    got = m.ssm_kv_page_select_fwd(q, b, big[:, :cols], c.t(lens), page_size=16, top_k=30, first=2, last=0, selected=out, workspace=ws)
    assert got.data_ptr() == out.data_ptr()
    np.testing.assert_array_equal(out.cpu().numpy(), longctx.page_select(n64(q), n64(b), c.table, lens, 16, 30, 2, 0))


# ------------------------------------------------------------- attention ----
def _lists(rng, lens, table, Hk, ps, top_k):
    """Lists as the choice gives them: rising places, all of them where they are few."""
    out = np.full((len(lens), Hk, top_k), -1)
    for r, n in enumerate(lens):
        n = -(-min(max(int(n), 0), table.shape[1] * ps) // ps)
        for g in range(Hk):
            out[r, g, :min(n, top_k)] = np.sort(rng.permutation(n)[:top_k])
    return out


def _attend(c, q, sel, lens, sc, **kw):
    return lib().ssm_select_attn_decode_fwd(q, c.k, c.v, c.t(c.table), c.t(lens), c.t(sel), scale=sc, k_scale=c.scale, v_scale=c.scale,
                                            return_lse=True, **kw)


def _check(name, c, q, sel, lens, sc, got=None):
    got = got or _attend(c, q, sel, lens, sc)
    k64, v64, H = c.k64(), c.v64(), q.shape[1]
    want = longctx.select_attn_decode(n64(q), k64, v64, c.table, lens, sel, sc)
    toks = [longctx._tokens(c.table[r], lens[r], c.ps, c.pages) for r in range(len(lens))]

    def rows_of(r, h):
        g = h * c.Hk // H
        held = -(-min(max(int(lens[r]), 0), c.table.shape[1] * c.ps) // c.ps)
        keep = set(int(x) for x in sel[r][g][:held])
        t = [x for x in toks[r] if x[0] // c.ps in keep]
        p, i = [x[1] for x in t], [x[2] for x in t]
        return k64[p, i, g], v64[p, i, g]

    worst = compare(got, want, rows_of, q, sc, c.cache != "f32", 0.0)
    report("select attention " + name, o_of_bound=worst[0], lse_of_bound=worst[1])
    assert worst[0] <= 1.0 and worst[1] <= 1.0, worst


ATTN = [  # lens, H, Hk, d, cache, page, layout, top_k
    (EDGES, 4, 2, 64, "bf16", 16, "nhd", 3), (EDGES, 4, 4, 128, "bf16", 1, "nhd", 40), (EDGES, 6, 2, 128, "bf16", 8, "hnd", 9),
    (EDGES, 5, 1, 80, "bf16", 24, "nhd", 5), (EDGES, 8, 1, 96, "bf16", 7, "hnd", 100), (EDGES, 2, 2, 192, "bf16", 64, "nhd", 2),
    (EDGES, 4, 1, 256, "bf16", 16, "nhd", 10), (EDGES, 17, 1, 128, "bf16", 16, "nhd", 7), (EDGES, 40, 2, 72, "bf16", 16, "nhd", 1),
    (EDGES, 8, 2, 128, "f8", 16, "nhd", 6), (EDGES, 8, 1, 64, "f8", 64, "hnd", 3), (EDGES, 4, 2, 192, "f8", 1, "nhd", 33),
    (EDGES, 2, 1, 256, "f8", 8, "nhd", 11), (EDGES, 5, 1, 256, "f32", 24, "nhd", 4), (EDGES, 4, 4, 128, "f32", 16, "hnd", 8),
    (EDGES, 20, 1, 64, "f32", 8, "nhd", 20), (EDGES, 2, 1, 72, "f32", 16, "nhd", 50),
    ([5000, 1, 3000, 0, 129], 8, 2, 128, "bf16", 16, "nhd", 130), ([20011], 4, 1, 64, "bf16", 64, "hnd", 200),
    ([9000], 8, 8, 64, "f8", 16, "nhd", 64), ([3001, 2000], 3, 1, 256, "f32", 16, "nhd", 100), ([100] * 300, 2, 2, 64, "bf16", 16, "nhd", 4),
    ([7000, 3, 900], 8, 4, 256, "bf16", 16, "nhd", 200), (list(range(71)) * 16, 4, 2, 64, "bf16", 16, "nhd", 2),
    ([2100] + [7] * 1050, 2, 2, 64, "bf16", 16, "hnd", 132), ([0, 2100, 64] * 350, 4, 2, 128, "f8", 16, "nhd", 70),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "%d-%d-H%d-%d-d%d-%s-p%d-%s-k%d" % ((len(c[0]), max(c[0])) + c[1:]))
def test_attention_against_the_oracle(cuda_device, case):
    lens, H, Hk, d, cache, ps, layout, top_k = case
    c = Paged(cuda_device, 80 + d, lens, Hk, d, cache, ps, layout)
    q = c.queries(len(lens), H, d)
    _check(str(case[1:]), c, q, _lists(c.rng, lens, c.table, Hk, ps, top_k), lens, d ** -0.5)


def test_lists_of_any_content(cuda_device):
    """Entries that are no page of the row, in any order, a page twice (counted twice), nothing at all, and pages outside
    the cache."""
    c = Paged(cuda_device, 81, [100, 200, 90, 64, 300], 2, 64, "bf16", 16)
    c.table[1, 3], c.table[1, 4] = -1, c.pages
    q = c.queries(5, 4, 64)
    sel = np.full((5, 2, 6), -1)
    sel[0, 0], sel[0, 1] = [6, -1, 0, 7, 1 << 30, 2], [-5, 1, 99, 3, -1, 0]
    sel[1, 0], sel[1, 1] = [3, 4, 5, 0, 12, 11], [12, 3, 4, -1, -1, -1]
    sel[2, 1] = [5, 4, 3, 2, 1, 0]
    sel[4, 0], sel[4, 1] = [2, 2, 2, 18, 18, 0], [7] * 6
    _check("any list", c, q, sel, c.lens, 0.2)


def test_attention_over_every_page_is_attention(cuda_device):
    """The same tokens as ssm_paged_attn_decode_fwd: both within their bounds of one value; and the same twice, on another
    stream, and into tensors of the caller's."""
    import torch
    m = lib()
    c = Paged(cuda_device, 82, [1000, 0, 77], 2, 128, "bf16", 16)
    q = c.queries(3, 8, 128)
    sel = np.tile(np.arange(c.table.shape[1]), (3, 2, 1))
    a = _attend(c, q, sel, c.lens, 0.09)
    b = m.ssm_paged_attn_decode_fwd(q, c.k, c.v, c.t(c.table), c.t(c.lens), scale=0.09, return_lse=True)
    assert (np.abs(n64(a[0]) - n64(b[0])) <= 2.0 ** -7 * np.abs(n64(b[0])) + 1e-5).all()
    np.testing.assert_allclose(n64(a[1]), n64(b[1]), atol=1e-5)
    ws = torch.full((m.ssm_select_attn_decode_fwd_workspace_size(3, 8, 2, 128, c.table.shape[1], 16, sel.shape[2]),), 255,
                    dtype=torch.uint8, device=cuda_device)
    o, lse = torch.empty_like(q), torch.empty((3, 8), device=cuda_device)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        got = _attend(c, q, sel, c.lens, 0.09, o=o, lse=lse, workspace=ws)
    other.synchronize()
    assert got[0].data_ptr() == o.data_ptr() and torch.equal(o, a[0]) and torch.equal(lse, a[1])


def test_no_rows(cuda_device):
    import torch
    i = lambda *n: torch.zeros(n, dtype=torch.int32, device=cuda_device)  # noqa: E731
    q, c = torch.zeros((0, 4, 64), device=cuda_device), torch.zeros((2, 16, 2, 64), device=cuda_device)
    assert lib().ssm_select_attn_decode_fwd(q, c, c.clone(), i(0, 3), i(0), i(0, 2, 4), scale=1.0).shape == (0, 4, 64)
    b = torch.zeros((2, 2, 2, 64), device=cuda_device)
    assert lib().ssm_kv_page_select_fwd(q, b, i(0, 3), i(0), page_size=16, top_k=2).shape == (0, 2, 2)


def test_a_decode_step_in_a_graph(cuda_device):
    """Bounds, choice and attention captured together; lengths, q and the new keys change between replays, with eager calls
    in between on copies of the same state."""
    import torch
    m = lib()
    c = Paged(cuda_device, 83, [600, 20, 333, 1], 2, 128, "bf16", 16, cols=40, spare=120, nan=False)
    table = c.t(np.random.default_rng(1).permutation(c.pages)[:160].reshape(4, 40))
    q, old, new = c.queries(4, 8, 128), c.t([0, 0, 0, 0]), c.t([600, 20, 333, 1])
    b = torch.zeros((c.pages, 2, 2, 128), dtype=torch.bfloat16, device=cuda_device)
    sel = torch.empty((4, 2, 8), dtype=torch.int32, device=cuda_device)
    o, lse = torch.empty_like(q), torch.empty((4, 8), device=cuda_device)
    ws1 = torch.empty(m.ssm_kv_page_select_fwd_workspace_size(4, 2, 40, 8), dtype=torch.uint8, device=cuda_device)
    ws2 = torch.empty(m.ssm_select_attn_decode_fwd_workspace_size(4, 8, 2, 128, 40, 16, 8), dtype=torch.uint8, device=cuda_device)

    def call():
        m.ssm_kv_page_bounds_update(c.k, b, table, old, new)
        m.ssm_kv_page_select_fwd(q, b, table, new, page_size=16, top_k=8, first=1, last=2, selected=sel, workspace=ws1)
        m.ssm_select_attn_decode_fwd(q, c.k, c.v, table, new, sel, scale=0.09, o=o, lse=lse, workspace=ws2)

    g = captured(call)
    for n0, n1 in (([0] * 4, [600, 20, 333, 1]), ([600, 20, 333, 1], [601, 0, 334, 640]), ([601, 0, 334, 640], [602, 300, 0, 640]),
                   ([0] * 4, [0] * 4), ([0] * 4, [640] * 4)):
        old.copy_(torch.tensor(n0))
        new.copy_(torch.tensor(n1))
        q.copy_(torch.randn_like(q))
        c.k.copy_(torch.randn_like(c.k))
        before = b.clone()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (b, sel, o, lse)]
        b.copy_(before)
        for t in (sel, o, lse):
            t.fill_(9)
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, (b, sel, o, lse)))
        want = longctx.page_select(n64(q), n64(b), table.cpu().numpy(), n1, 16, 8, 1, 2)
        np.testing.assert_array_equal(sel.cpu().numpy(), want)
