"""ssm_paged_attn_decode_fwd on the GPU against the fp64 oracle.

Bounds, derived from the arithmetic (u = 2^-24): a score is a sum of d products (exact in
fp32 for bf16 and 8-bit values) with at most d roundings, so within (d + 4) u of scale *
sum |q k|, and as the exponent of 2 it is rounded once more, u |s| log2 e; call the largest
of a head D.  Every exponential is then within 2 D + 4 u of itself, and their sum within n u more
for n tokens.  The quotient is a weighted mean of v, so its error is at most twice that of
the weights times the largest |v|; p as two bf16 values adds 2^-17 (only where v is not fp32), and the output's own
rounding 2^-8 |o| (bf16) or u |o|.  lse is within the weights' error of its own value."""
import numpy as np
import pytest

from helpers import lib, report
from oracle import paged

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _make(device, seed, lens, H, Hk, d, cache, ps, layout, cols=None, spare=3, nan=True):
    import torch
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    have = -(-np.maximum(lens, 0) // ps)
    cols = cols or max(1, int(have.max()))
    have = np.minimum(have, cols)
    total = int(have.sum()) + spare
    table = np.full((len(lens), cols), -1)
    table[np.arange(cols)[None] < have[:, None]] = rng.permutation(total)[:have.sum()]
    dt = {"bf16": torch.bfloat16, "f8": torch.float8_e4m3fn, "f32": torch.float32}[cache]
    qt = torch.float32 if cache == "f32" else torch.bfloat16
    scale = 0.03 if cache == "f8" else 1.0
    q = torch.tensor(rng.standard_normal((len(lens), H, d)), device=device).to(qt)
    caches = []
    for _ in range(2):
        c = torch.tensor(rng.standard_normal((total, ps, Hk, d)) / scale, dtype=torch.float32)
        if nan:       # what no request holds: NaN
            used = np.zeros((total, ps), bool)
            for r, n in enumerate(lens):
                j = np.arange(min(max(int(n), 0), cols * ps))
                used[table[r, j // ps], j % ps] = True
            c[torch.tensor(~used)] = float("nan")
        c = c.to(dt)
        if layout == "hnd":
            c = c.view(torch.uint8 if cache == "f8" else dt).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3).view(dt)
        caches.append(c.to(device))
    return q, caches[0], caches[1], table, lens, scale


def _n(t):
    return t.detach().float().double().cpu().numpy()


def _compare(name, got, q, kc, vc, table, lens, sc, cache_scale, window=0):
    o, lse = got
    k64, v64 = _n(kc) * cache_scale, _n(vc) * cache_scale
    want, wlse = paged.paged_attn_decode(_n(q), k64, v64, table, lens, sc, window)
    B, H, d = want.shape
    Hk, ps = kc.shape[2], kc.shape[1]
    bf = str(o.dtype) == "torch.bfloat16"
    worst = [0.0, 0.0]
    assert (np.isneginf(_n(lse)) == np.isneginf(wlse)).all()
    assert o.isfinite().all()
    for r in range(B):
        n = min(max(int(lens[r]), 0), table.shape[1] * ps)
        j = np.arange(max(0, n - window) if window else 0, n)
        pg = table[r, j // ps] if len(j) else np.zeros(0, int)
        ok = (pg >= 0) & (pg < kc.shape[0])
        j, pg = j[ok], pg[ok]
        if not len(j):
            assert (o[r] == 0).all()
            continue
        for h in range(H):
            k, v = k64[pg, j % ps, h * Hk // H], v64[pg, j % ps, h * Hk // H]
            s = abs(sc) * (np.abs(k) @ np.abs(_n(q)[r, h])).max()
            D = (d + 4) * U * s + 2 * U * s
            werr = 2 * D + 4 * U + len(j) * U + (2.0 ** -17 if bf else 0)
            tol = 2 * werr * np.abs(v).max() + (2.0 ** -8 if bf else U) * np.abs(want[r, h])
            worst[0] = max(worst[0], float((np.abs(_n(o)[r, h] - want[r, h]) / tol).max()))
            worst[1] = max(worst[1], abs(_n(lse)[r, h] - wlse[r, h]) / (werr + 4 * U * abs(wlse[r, h])))
    report(name, o_of_bound=worst[0], lse_of_bound=worst[1])
    assert worst[0] <= 1.0 and worst[1] <= 1.0, (name, worst)


def _run(device, q, kc, vc, table, lens, sc, scale, window=0, **kw):
    import torch
    return lib().ssm_paged_attn_decode_fwd(q, kc, vc, torch.tensor(table, dtype=torch.int32, device=device),
                                           torch.tensor(lens, dtype=torch.int32, device=device), scale=sc, window=window,
                                           k_scale=scale, v_scale=scale, return_lse=True, **kw)


EDGES = [1, 0, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400, -3]
CASES = [  # lens, H, Hk, d, cache, page, layout, window
    ([1], 1, 1, 64, "bf16", 16, "nhd", 0),
    (EDGES, 4, 2, 64, "bf16", 16, "nhd", 0),
    (EDGES, 4, 4, 128, "bf16", 1, "nhd", 0),
    (EDGES, 6, 2, 128, "bf16", 8, "hnd", 0),
    (EDGES, 5, 1, 80, "bf16", 24, "nhd", 0),
    (EDGES, 8, 1, 96, "bf16", 7, "hnd", 33),
    (EDGES, 2, 2, 192, "bf16", 64, "nhd", 0),
    (EDGES, 4, 1, 256, "bf16", 16, "nhd", 100),
    (EDGES, 16, 1, 128, "bf16", 16, "nhd", 1),
    (EDGES, 17, 1, 128, "bf16", 16, "nhd", 0),          # two passes over the heads
    (EDGES, 40, 2, 72, "bf16", 16, "nhd", 50),
    (EDGES, 3, 1, 8, "bf16", 5, "nhd", 0),
    (EDGES, 8, 2, 128, "f8", 16, "nhd", 0),
    (EDGES, 8, 1, 64, "f8", 64, "hnd", 0),
    (EDGES, 5, 1, 96, "f8", 24, "hnd", 77),
    (EDGES, 4, 2, 192, "f8", 1, "nhd", 0),
    (EDGES, 2, 1, 256, "f8", 8, "nhd", 0),
    (EDGES, 6, 2, 16, "f8", 16, "nhd", 0),
    (EDGES, 5, 1, 256, "f32", 24, "nhd", 0),
    (EDGES, 4, 4, 128, "f32", 16, "hnd", 31),
    (EDGES, 20, 1, 64, "f32", 8, "nhd", 0),
    (EDGES, 3, 3, 192, "f32", 1, "nhd", 0),
    (EDGES, 2, 1, 72, "f32", 16, "nhd", 0),
    ([5000, 1, 3000, 0, 129], 8, 2, 128, "bf16", 16, "nhd", 0),
    ([20011], 4, 1, 64, "bf16", 64, "hnd", 0),           # one row over every block
    ([9000, 8000], 8, 1, 128, "f8", 64, "hnd", 4097),
    ([3001, 2000], 3, 1, 256, "f32", 16, "nhd", 0),
    ([100] * 300, 2, 2, 64, "bf16", 16, "nhd", 0),       # more rows than a block has threads
    # kv heads side by side (their rows share cache lines, or are wide), rows over many blocks too
    (EDGES + [3000], 8, 4, 80, "bf16", 16, "nhd", 0),
    (EDGES + [9000], 8, 8, 64, "f8", 16, "nhd", 0),
    ([20000, 3], 6, 6, 96, "f8", 24, "nhd", 10001),
    ([7000, 3, 900], 8, 4, 256, "bf16", 16, "nhd", 0),
    ([5000, 1], 6, 2, 192, "f32", 16, "nhd", 0),
    # a (row, kv head) for every wave of the chip: blocks of one wave
    (list(range(71)) * 16, 4, 2, 64, "bf16", 16, "nhd", 0),
    (list(range(0, 280, 4)) * 8, 4, 4, 96, "bf16", 8, "nhd", 90),
    (list(range(3, 143, 2)) * 8, 4, 4, 128, "f8", 64, "hnd", 0),
    ([5, 0, 700] * 120, 6, 3, 256, "f32", 16, "nhd", 0),
    ([2000] + [1] * 1100, 2, 2, 128, "f32", 16, "nhd", 0),
    # short rows, a block for each (row, kv head): by the window alone, in two passes, side by side
    (EDGES + [7000], 4, 2, 128, "bf16", 16, "nhd", 300),
    (EDGES + [7000], 34, 2, 128, "bf16", 24, "hnd", 300),
    (EDGES, 6, 6, 80, "bf16", 7, "nhd", 257),
    ([100, 0, 31, 384], 40, 1, 128, "bf16", 16, "nhd", 0),
    (EDGES, 8, 4, 192, "f32", 16, "nhd", 150),
    (list(range(0, 600, 5)) * 2, 2, 1, 72, "bf16", 1, "nhd", 0),
    (list(range(40, 440)) + [0], 6, 3, 256, "bf16", 16, "nhd", 0),
    # and rows too long for that, on blocks of one wave
    ([2100] + [7] * 1050, 2, 2, 64, "bf16", 16, "hnd", 0),
    ([0, 2100, 64] * 350, 4, 2, 128, "f8", 16, "nhd", 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%d-%d-H%d-%d-d%d-%s-p%d-%s-w%d" % ((len(c[0]), max(c[0])) + c[1:]))
def test_against_the_oracle(cuda_device, case):
    lens, H, Hk, d, cache, ps, layout, window = case
    q, kc, vc, table, lens, s = _make(cuda_device, 10 + d, lens, H, Hk, d, cache, ps, layout)
    sc = d ** -0.5
    got = _run(cuda_device, q, kc, vc, table, lens, sc, s, window)
    _compare("attn %s" % (case[1:],), got, q, kc, vc, table, lens, sc, s, window)


@pytest.mark.parametrize("H,Hk,d,cache,layout,window", [
    (8, 2, 128, "bf16", "nhd", 0), (2, 2, 64, "bf16", "hnd", 0), (20, 1, 80, "bf16", "nhd", 0), (8, 4, 96, "f8", "nhd", 0),
    (8, 8, 128, "f8", "hnd", 3333), (6, 3, 128, "f32", "nhd", 0), (10, 2, 256, "f32", "nhd", 2000), (8, 4, 256, "bf16", "nhd", 0)])
def test_one_row_in_a_wide_table(cuda_device, H, Hk, d, cache, layout, window):
    """One request, of any length, in a table for 6400 tokens (fewer tokens than blocks, too), with a
    workspace that holds NaN before the call: what no block wrote is not used."""
    import torch
    m = lib()
    ws = torch.empty(m.ssm_paged_attn_decode_fwd_workspace_size(1, H, Hk, d, 400, 16), dtype=torch.uint8, device=cuda_device)
    for n in (0, 1, 17, 130, 700, 3001, 6400):
        q, kc, vc, table, lens, s = _make(cuda_device, 20 + n, [n], H, Hk, d, cache, 16, layout, cols=400)
        ws.fill_(255)
        got = _run(cuda_device, q, kc, vc, table, lens, d ** -0.5, s, window, workspace=ws)
        _compare("attn one row %s" % ((n, H, Hk, d, cache, window),), got, q, kc, vc, table, lens, d ** -0.5, s, window)
    table[0, 100:300] = -1                      # whole pieces without a page in the cache
    got = _run(cuda_device, q, kc, vc, table, lens, d ** -0.5, s, window, workspace=ws)
    _compare("attn one row, pages missing", got, q, kc, vc, table, lens, d ** -0.5, s, window)


def test_twice_the_same_and_without_lse(cuda_device):
    import torch
    q, kc, vc, table, lens, s = _make(cuda_device, 3, [700, 33, 2100], 8, 2, 128, "bf16", 16, "nhd")
    a = _run(cuda_device, q, kc, vc, table, lens, 0.1, s)
    b = _run(cuda_device, q, kc, vc, table, lens, 0.1, s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    o = lib().ssm_paged_attn_decode_fwd(q, kc, vc, torch.tensor(table, dtype=torch.int32, device=cuda_device),
                                        torch.tensor(lens, dtype=torch.int32, device=cuda_device), scale=0.1)
    assert torch.equal(o, a[0])


def test_pages_outside_the_cache_are_left_out(cuda_device):
    q, kc, vc, table, lens, s = _make(cuda_device, 4, [200, 90, 64], 4, 2, 64, "bf16", 16, "nhd")
    table[0, 3], table[0, 5], table[2, :] = -1, kc.shape[0], 1 << 30
    got = _run(cuda_device, q, kc, vc, table, lens, 0.2, s)
    _compare("attn bad pages", got, q, kc, vc, table, lens, 0.2, s)


def test_lens_past_the_table(cuda_device):
    q, kc, vc, table, lens, s = _make(cuda_device, 5, [90, 100000, 50], 4, 2, 64, "bf16", 16, "nhd", cols=6)
    got = _run(cuda_device, q, kc, vc, table, lens, 0.2, s)
    _compare("attn long lens", got, q, kc, vc, table, lens, 0.2, s)


def test_scores_of_every_size(cuda_device):
    """Scores of hundreds, a negative scale, and rows of equal keys: the maximum is kept and
    nothing overflows."""
    for sc in (8.0, -8.0, 0.0):
        q, kc, vc, table, lens, s = _make(cuda_device, 6, [300, 40], 4, 2, 64, "f32", 16, "nhd")
        _compare("attn scale %g" % sc, _run(cuda_device, q, kc, vc, table, lens, sc, s), q, kc, vc, table, lens, sc, s)


def test_infinite_scores(cuda_device):
    """-inf scores weigh nothing; a row of only those is empty; NaN and +inf scores give NaN."""
    import torch
    q, kc, vc, table, lens, s = _make(cuda_device, 7, [40, 40, 40, 40], 2, 1, 64, "f32", 16, "nhd")
    q = q.abs() + 0.1
    rows = [[(int(table[r, j // 16]), j % 16) for j in range(40)] for r in range(4)]
    for p, i in rows[0][3:20]:
        kc[p, i, 0, 5] = -float("inf")
    for p, i in rows[1]:
        kc[p, i, 0, 7] = -float("inf")
    kc[rows[2][11]][0, 0] = float("nan")
    kc[rows[3][39]][0, 0] = float("inf")
    o, lse = _run(cuda_device, q, kc, vc, table, lens, 0.125, s)
    keep = torch.tensor([j for j in range(40) if not 3 <= j < 20])
    k = torch.stack([kc[p, i, 0] for p, i in rows[0]])[keep].double()
    v = torch.stack([vc[p, i, 0] for p, i in rows[0]])[keep].double()
    sc = 0.125 * q[0].double() @ k.T
    # 23 scores of about 20: within 1e-5 by the bounds above
    assert (o[0].double() - torch.softmax(sc, -1) @ v).abs().max() <= 2e-4
    assert (lse[0].double() - torch.logsumexp(sc, -1)).abs().max() <= 2e-4
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    assert o[2].isnan().all() and lse[2].isnan().all() and o[3].isnan().all() and lse[3].isnan().all()


def test_strided_q_shared_pages_and_outputs_given(cuda_device):
    """The tokens of a prompt as rows with growing lens over one request's pages, q a slice of
    a projection, a table with a longer row stride, and o, lse, workspace of the caller."""
    import torch
    m = lib()
    q, kc, vc, table, lens, s = _make(cuda_device, 8, [70], 6, 2, 128, "bf16", 16, "nhd")
    T = 70
    rng = np.random.default_rng(9)
    proj = torch.tensor(rng.standard_normal((T, 1000 + 24)), device=cuda_device).to(torch.bfloat16)
    q = proj[:, 256:].view(T, 6, 128)
    big = torch.full((T, 9), -1, dtype=torch.int32, device=cuda_device)
    big[:, :table.shape[1]] = torch.tensor(table, dtype=torch.int32)
    t = big[:, :table.shape[1]]
    lens = np.arange(1, T + 1)
    o = torch.empty((T, 6, 128), dtype=torch.bfloat16, device=cuda_device)
    lse = torch.empty((T, 6), device=cuda_device)
    ws = torch.empty(m.ssm_paged_attn_decode_fwd_workspace_size(T, 6, 2, 128, table.shape[1], 16), dtype=torch.uint8,
                     device=cuda_device)
    got = m.ssm_paged_attn_decode_fwd(q, kc, vc, t, torch.tensor(lens, dtype=torch.int32, device=cuda_device), scale=0.09,
                                      o=o, lse=lse, workspace=ws)
    assert got[0].data_ptr() == o.data_ptr() and got[1].data_ptr() == lse.data_ptr()
    _compare("attn prompt rows", got, q, kc, vc, np.repeat(table, T, 0), lens, 0.09, s)


def test_no_rows(cuda_device):
    import torch
    q = torch.zeros((0, 4, 64), device=cuda_device)
    c = torch.zeros((2, 16, 2, 64), device=cuda_device)
    i = lambda *n: torch.zeros(n, dtype=torch.int32, device=cuda_device)  # noqa: E731
    o, lse = lib().ssm_paged_attn_decode_fwd(q, c, c.clone(), i(0, 3), i(0), scale=1.0, return_lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_a_cache_past_4_gib(cuda_device):
    """Offsets past 32 bits: pages at the end of a cache of 5 GiB a tensor."""
    import torch
    P, ps, Hk, d = 163840, 16, 8, 128
    kc, vc = (torch.zeros((P, ps, Hk, d), dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    rng = np.random.default_rng(10)
    last = [P - 1, P - 40000, P - 3, 131072, 131071]
    for c in (kc, vc):
        for p in last:
            c[p] = torch.tensor(rng.standard_normal((ps, Hk, d)), device=cuda_device).to(torch.bfloat16)
    q = torch.tensor(rng.standard_normal((1, 16, d)), device=cuda_device).to(torch.bfloat16)
    got = _run(cuda_device, q, kc, vc, np.array([last]), [77], 0.09, 1.0)
    _compare("attn 5 GiB", got, q, kc[last], vc[last], np.array([[0, 1, 2, 3, 4]]), [77], 0.09, 1.0)


@pytest.mark.parametrize("H,Hk,d", [(8, 2, 128), (16, 1, 256), (4, 2, 64)])     # 65 KiB of LDS a block; a block a head
def test_in_a_graph_with_lens_and_table_changing(cuda_device, H, Hk, d):
    """Captured once; lens, table and q change in place between replays.  The grid depends on
    the table's size alone, so every replay has to equal the eager call."""
    import torch
    m = lib()
    q, kc, vc, table, lens, s = _make(cuda_device, 11, [600, 20, 333, 1], H, Hk, d, "bf16", 16, "nhd", nan=False)
    t = torch.tensor(table, dtype=torch.int32, device=cuda_device)
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    o, lse = torch.empty_like(q), torch.empty((4, H), device=cuda_device)
    ws = torch.empty(m.ssm_paged_attn_decode_fwd_workspace_size(4, H, Hk, d, t.shape[1], 16), dtype=torch.uint8, device=cuda_device)
    call = lambda: m.ssm_paged_attn_decode_fwd(q, kc, vc, t, n, scale=0.09, o=o, lse=lse, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    t[:] = torch.arange(t.numel(), device=cuda_device).view(t.shape) % kc.shape[0]
    for new in ([600, 20, 333, 1], [0, 608, 1, 5], [300, 301, 302, 303], [0, 0, 0, 0]):
        n.copy_(torch.tensor(new))
        q.copy_(torch.randn_like(q))
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        a, b = o.clone(), lse.clone()
        o.fill_(9.0)
        call()
        torch.cuda.synchronize()
        assert torch.equal(a, o) and torch.equal(b, lse)


@pytest.mark.parametrize("H,Hk,d,cache,cols", [(8, 2, 128, "bf16", 1), (4, 4, 64, "bf16", 1), (2, 1, 256, "bf16", 1), (17, 1, 192, "bf16", 1),
                                               (8, 2, 128, "f8", 1), (4, 2, 64, "f8", 1), (3, 1, 256, "f8", 1), (4, 2, 128, "f32", 1),
                                               (8, 2, 128, "bf16", 4000), (8, 2, 128, "f8", 4000)])
def test_the_weights_bits_cancel_where_v_does(cuda_device, H, Hk, d, cache, cols):
    """Three tokens with scores 0, t and t + e, |e| <= 2^-12, and v = 0, 1 and -1: o = (p1 - p2) / (1 + p1 + p2) is about
    2^-14, so the output's own rounding is under 2^-21 and a weight that lost its last bits shows.  (Two bf16
    values in place of a weight are up to 2^-18 off, o up to 2^-18.) Every product and both scores are
    exact in fp32; a weight under 1/2 takes (2 |s| + 4) u of itself from its exponent and the exponential, two of
    them 5 u of o, and adding them up in fp32 8 u of the sum of weights at most, 5 u of o: within 12 u."""
    import torch
    B = 300 if cols == 1 else 40
    rng = np.random.default_rng(31)
    dt = {"bf16": torch.bfloat16, "f8": torch.float8_e4m3fn, "f32": torch.float32}[cache]
    q = torch.zeros((B, H, d))
    q[..., 0] = torch.tensor(-rng.uniform(0.7, 1.0, (B, H)))
    q[..., 1] = torch.tensor(rng.uniform(2.0 ** -13, 2.0 ** -12, (B, H)) * rng.choice([-1, 1], (B, H)))
    q = q.to(torch.float32 if cache == "f32" else torch.bfloat16).to(cuda_device)
    kc, vc = torch.zeros((1, 16, Hk, d)), torch.zeros((1, 16, Hk, d))
    kc[0, 1:3, :, 0], kc[0, 2, :, 1] = 1.0, 1.0
    vc[0, 1], vc[0, 2] = 1.0, -1.0
    kc, vc = kc.to(dt).to(cuda_device), vc.to(dt).to(cuda_device)
    o, _ = _run(cuda_device, q, kc, vc, np.zeros((B, cols)), [3] * B, 1.0, 1.0)
    t, e = _n(q)[..., 0], _n(q)[..., 1]
    want = (np.exp(t) - np.exp(t + e)) / (1 + np.exp(t) + np.exp(t + e))
    tol = (U if cache == "f32" else 2.0 ** -8) * np.abs(want) + 12 * U
    worst = float((np.abs(_n(o) - want[..., None]) / tol[..., None]).max())
    report("attn weights %s" % ((H, Hk, d, cache, cols),), of_bound=worst)
    assert worst <= 1.0


def test_lse_does_not_hold_a_large_output(cuda_device):
    """lse kept for a later join: its memory is its own where o is over 4 MiB."""
    import torch
    for B in (20, 4000):
        q, kc, vc, table, lens, s = _make(cuda_device, 12, [3] * B, 8, 2, 128, "bf16", 16, "nhd")
        o, lse = _run(cuda_device, q, kc, vc, table, lens, 0.1, s)
        assert lse.untyped_storage().nbytes() <= (B * 8 * 4 + 512 if B == 4000 else (4 << 20) + B * 8 * 4 + 512)
        a, _ = _run(cuda_device, q, kc, vc, table, lens, 0.1, s, o=torch.empty_like(q))
        assert torch.equal(a, o)


LSE_CASES = [CASES[i] for i in (1, 5, 9, 12, 16, 18, 23, 24, 28, 30, 34, 37, 39, 43)] + [([n], 8, 2, 128, c, 16, "nhd", 0) for n in (0, 1, 700, 6400) for c in ("bf16", "f8", "f32")]


@pytest.mark.parametrize("case", LSE_CASES, ids=lambda c: "%d-%d-H%d-%d-d%d-%s-p%d-%s-w%d" % ((len(c[0]), max(c[0])) + c[1:]))
def test_lse_is_finite_where_it_should_be(cuda_device, case):
    """lse alone, with a workspace that holds NaN before the call: -inf where a row has no token and nowhere else,
    finite elsewhere, and all of it within its bound (a NaN is within none)."""
    import torch
    lens, H, Hk, d, cache, ps, layout, window = case
    q, kc, vc, table, lens, s = _make(cuda_device, 60 + d, lens, H, Hk, d, cache, ps, layout, cols=400 if len(lens) == 1 and lens[0] < 7000 else None)
    ws = torch.full((lib().ssm_paged_attn_decode_fwd_workspace_size(len(lens), H, Hk, d, table.shape[1], ps),), 255, dtype=torch.uint8,
                    device=cuda_device)
    sc = d ** -0.5
    got = _n(_run(cuda_device, q, kc, vc, table, lens, sc, s, window, workspace=ws)[1])
    k64 = _n(kc) * s
    _, want = paged.paged_attn_decode(_n(q), k64, _n(vc) * s, table, lens, sc, window)
    assert (np.isfinite(got) == np.isfinite(want)).all() and (np.isneginf(got) == np.isneginf(want)).all()
    n = np.minimum(np.maximum(lens, 0), table.shape[1] * ps)[:, None]
    # |s| <= scale |k| |q| of the largest cached row (rows that no request holds are NaN)
    big = abs(sc) * np.sqrt(np.nan_to_num((k64 ** 2).sum(-1)).max()) * np.sqrt((_n(q) ** 2).sum(-1))
    tol = 2 * (d + 6) * U * big + 4 * U + n * U + 4 * U * np.abs(np.where(np.isfinite(want), want, 0.0))
    there = np.isfinite(want)
    ratio = np.abs(got[there] - want[there]) / tol[there]
    report("attn lse %s" % (case[1:],), of_bound=float(ratio.max()) if ratio.size else 0.0)
    assert (ratio <= 1.0).all()
