"""ssm_qk_norm_rope_fwd, _bwd and _cache_fwd on the GPU against the fp64 oracle.

Bounds, derived from the arithmetic (u = 2^-24, the largest rounding of one fp32 operation):
a norm's sum has at most 22 roundings in a row (16 of a lane, 6 across lanes), halved by
the root; root, quotient, mean and two products add 5; a cosine or sine is within 3 u, so
a rotated value is within 6 u of its pair's size, and 2 u for its own products: under
32 u (|a| + |b|) in all, a and b the pair before the turn.  A bf16 result adds half a step,
2^-8 of it; an e4m3 one 2^-4 of it, or 2^-10 (half the smallest step) where it is tiny."""
import numpy as np
import pytest

from helpers import lib, report
from oracle import paged

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
K = 32 * U


def _pair(y, rot, il):
    """|a| + |b| of each value's pair (the value alone past rot)."""
    m = np.abs(y)
    a, b = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if il else (np.arange(rot // 2), np.arange(rot // 2, rot))
    s = m[..., a] + m[..., b]
    m[..., a], m[..., b] = s, s
    return m


def _make(case, device, seed):
    import torch
    T, H, Hk, d, rot, dtype, il, norm = case
    rng = np.random.default_rng(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    t = lambda a: torch.tensor(np.asarray(a, np.float32), device=device).to(dt)  # noqa: E731
    qkv = t(rng.standard_normal((T, (H + 2 * Hk) * d)))
    q, k, v = qkv[:, :H * d].view(T, H, d), qkv[:, H * d:(H + Hk) * d].view(T, Hk, d), qkv[:, (H + Hk) * d:].view(T, Hk, d)
    w = [torch.tensor(rng.normal(1, 0.1, d), dtype=torch.float32, device=device) if norm else None for _ in range(2)]
    f = torch.tensor(1e6 ** (-np.arange(rot // 2) / max(1, rot // 2)), dtype=torch.float32, device=device)
    pos = torch.tensor(rng.integers(0, 131072) + np.arange(T), dtype=torch.int32, device=device)
    m = lib()
    flags = (m.SSM_ROPE_INTERLEAVED if il else 0) | (0 if norm else m.SSM_QK_NO_NORM)
    g = [t(rng.standard_normal((T, n, d))) for n in (H, Hk)]
    return q, k, v, w, f, pos, g, flags


def _n(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _check(name, got, want, tol):
    err = np.abs(_n(got) - want)
    assert got.isfinite().all()
    worst = float((err / np.maximum(tol, 1e-30)).max()) if err.size else 0.0
    report(name, of_bound=worst)
    assert worst <= 1.0, (name, worst)


SHAPES = [  # T, H, Hk, d, rot, dtype, interleaved, norm
    (1, 1, 1, 64, 64, "bf16", False, True),
    (5, 4, 2, 128, 128, "bf16", False, True),
    (67, 32, 8, 128, 128, "bf16", False, True),
    (300, 6, 3, 128, 64, "bf16", True, True),
    (33, 5, 1, 256, 128, "bf16", False, True),
    (40, 8, 8, 80, 40, "bf16", False, True),
    (31, 3, 3, 72, 24, "bf16", True, True),
    (129, 2, 1, 96, 96, "bf16", False, False),
    (17, 7, 1, 64, 0, "bf16", False, True),
    (9, 3, 1, 31, 10, "bf16", False, True),         # odd head: one element at a time
    (1021, 6, 3, 72, 24, "f32", True, True),
    (50, 4, 4, 256, 256, "f32", False, True),
    (64, 16, 2, 128, 32, "f32", False, False),
    (11, 2, 1, 255, 102, "f32", True, True),
    (6, 40, 1, 8, 8, "f32", False, True),
    (3, 2, 1, 1, 0, "f32", False, True),
    (700, 300, 7, 64, 64, "bf16", False, True),     # more heads than a block has lane groups
    (2000, 20, 4, 128, 64, "bf16", False, True),    # a token's heads in parts, more of them than waves
]
_id = lambda c: "T%d-H%d-%d-d%d-r%d-%s-%d%d" % c  # noqa: E731


@pytest.mark.parametrize("case", SHAPES, ids=_id)
def test_forward(cuda_device, case):
    T, H, Hk, d, rot, dtype, il, norm = case
    q, k, v, w, f, pos, _, flags = _make(case, cuda_device, 1)
    qo, ko = lib().ssm_qk_norm_rope_fwd(q, k, w[0], w[1], f, pos, flags=flags)
    for n, x, wx, y in (("q", q, w[0], qo), ("k", k, w[1], ko)):
        assert y.dtype == x.dtype and y.is_contiguous()
        want = paged.qk_norm_rope(_n(x), _n(wx), _n(f), _n(pos), interleaved=il)
        flat = paged.qk_norm_rope(_n(x), _n(wx), _n(f), 0 * _n(pos), interleaved=il)
        _check("rope %s %s" % (n, case), y, want, K * _pair(flat, rot, il) + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0))


@pytest.mark.parametrize("case", SHAPES, ids=_id)
def test_backward(cuda_device, case):
    T, H, Hk, d, rot, dtype, il, norm = case
    q, k, v, w, f, pos, g, flags = _make(case, cuda_device, 2)
    got = lib().ssm_qk_norm_rope_bwd(q, k, w[0], w[1], f, pos, g[0], g[1], flags=flags)
    for n, x, wx, gx in (("q", q, w[0], g[0]), ("k", k, w[1], g[1])):
        dx, dw = paged.qk_norm_rope_bwd(_n(x), _n(wx), _n(f), _n(pos), _n(gx), interleaved=il)
        size = _pair(np.abs(_n(gx)), rot, il)                      # of the cotangent, before and after its turn
        if norm:
            r = 1.0 / np.sqrt((_n(x) ** 2).mean(-1, keepdims=True) + 1e-6)
            wg, nx = np.abs(_n(wx)) * size, np.abs(_n(x)) * r
            size = r * (wg + nx * (wg * nx).mean(-1, keepdims=True))
        # 40: the 32 of a normed and turned value, and the mean's own 22 roundings over two factors
        tol = 64 * U * size + (2.0 ** -8 * np.abs(dx) if dtype == "bf16" else 0)
        _check("rope d%s %s" % (n, case), got["d" + n], dx, tol)
        if norm:
            # every term within 40 u of its size; chains of at most 128 additions before fp64
            terms = (_pair(np.abs(_n(gx)), rot, il) * nx).sum((0, 1))
            _check("rope dw%s %s" % (n, case), got["dw" + n], dw, (40 + 128) * U * terms)
        else:
            assert got["dw" + n] is None


def test_backward_many_tokens_and_twice_the_same(cuda_device):
    case = (4100, 8, 2, 128, 128, "bf16", False, True)
    import torch
    q, k, v, w, f, pos, g, flags = _make(case, cuda_device, 3)
    a = lib().ssm_qk_norm_rope_bwd(q, k, w[0], w[1], f, pos, g[0], g[1])
    b = lib().ssm_qk_norm_rope_bwd(q, k, w[0], w[1], f, pos, g[0], g[1])
    for n in a:
        assert torch.equal(a[n], b[n])
    for n, x, wx, gx in (("q", q, w[0], g[0]), ("k", k, w[1], g[1])):
        _, dw = paged.qk_norm_rope_bwd(_n(x), _n(wx), _n(f), _n(pos), _n(gx))
        nx = np.abs(_n(x)) / np.sqrt((_n(x) ** 2).mean(-1, keepdims=True) + 1e-6)
        _check("rope dw%s 4100" % n, a["dw" + n], dw, (40 + 128) * U * (_pair(np.abs(_n(gx)), 128, False) * nx).sum((0, 1)))


def test_backward_against_differences(cuda_device):
    """<dx, e> and <dw, e> against central differences of the forward along random e, fp32.
    A step of h = 2^-7 leaves a third-order term of about h^2 / 6 of the first-order size
    (1e-5) and a rounding of 32 u ||y|| ||g|| / h of its own; the bound takes 1e-3 of ||g|| ||e||."""
    import torch
    case = (37, 4, 2, 80, 40, "f32", False, True)
    q, k, v, w, f, pos, g, flags = _make(case, cuda_device, 4)
    m, h = lib(), 2.0 ** -7
    got = m.ssm_qk_norm_rope_bwd(q, k, w[0], w[1], f, pos, g[0], g[1])
    fwd = lambda q_, k_, w0, w1: m.ssm_qk_norm_rope_fwd(q_, k_, w0, w1, f, pos)  # noqa: E731
    gen = torch.Generator(device=cuda_device).manual_seed(5)
    for n in ("q", "k", "wq", "wk"):
        args = [q, k, w[0], w[1]]
        i = ("q", "k", "wq", "wk").index(n)
        e = torch.randn(args[i].shape, generator=gen, device=cuda_device)
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + h * e, args[i] - h * e
        side = i % 2
        diff = (fwd(*hi)[side].double() - fwd(*lo)[side].double()) / (2 * h)
        want = float((diff * g[side].double()).sum())
        have = float((got["d" + n].double() * e.double()).sum())
        bound = 1e-3 * float(g[side].double().norm() * e.double().norm())
        report("rope differences " + n, err=abs(want - have), bound=bound)
        assert abs(want - have) <= bound


@pytest.mark.parametrize("case", [(33, 3, 1, 128, 64, "bf16", False, True), (5, 6, 3, 72, 24, "f32", True, True),
                                  (7, 1, 1, 31, 10, "f32", False, True)], ids=_id)
def test_backward_without_an_eps(cuda_device, case):
    """eps = 0 where heads do not fill a wave's lanes: the idle lanes' 1/0 stays out of dw.
    Bounds as above."""
    T, H, Hk, d, rot, dtype, il, norm = case
    q, k, v, w, f, pos, g, flags = _make(case, cuda_device, 12)
    got = lib().ssm_qk_norm_rope_bwd(q, k, w[0], w[1], f, pos, g[0], g[1], eps=0.0, flags=flags)
    for n, x, wx, gx in (("q", q, w[0], g[0]), ("k", k, w[1], g[1])):
        dx, dw = paged.qk_norm_rope_bwd(_n(x), _n(wx), _n(f), _n(pos), _n(gx), eps=0.0, interleaved=il)
        r = 1.0 / np.sqrt((_n(x) ** 2).mean(-1, keepdims=True))
        size = _pair(np.abs(_n(gx)), rot, il)
        wg, nx = np.abs(_n(wx)) * size, np.abs(_n(x)) * r
        _check("rope eps 0 dw%s %s" % (n, case), got["dw" + n], dw, (40 + 128) * U * (size * nx).sum((0, 1)))
        size = r * (wg + nx * (wg * nx).mean(-1, keepdims=True))
        _check("rope eps 0 d%s %s" % (n, case), got["d" + n], dx, 64 * U * size + (2.0 ** -8 * np.abs(dx) if dtype == "bf16" else 0))


def test_in_place_q_alone_and_odd_views(cuda_device):
    import torch
    m = lib()
    case = (21, 4, 2, 64, 64, "bf16", False, True)
    q, k, v, w, f, pos, g, flags = _make(case, cuda_device, 6)
    qo, ko = m.ssm_qk_norm_rope_fwd(q, k, w[0], w[1], f, pos)
    qc, kc = q.contiguous(), k.contiguous()
    a, b = m.ssm_qk_norm_rope_fwd(qc, kc, w[0], w[1], f, pos, q_out=qc, k_out=kc)
    assert a.data_ptr() == qc.data_ptr() and torch.equal(a, qo) and torch.equal(b, ko)
    a, b = m.ssm_qk_norm_rope_fwd(q, None, w[0], None, f, pos)
    assert b is None and torch.equal(a, qo)
    # a view that starts at an odd element: one element at a time, the same values
    odd = torch.zeros(21 * 4 * 64 + 1, dtype=torch.bfloat16, device=cuda_device)[1:].view(21, 4, 64)
    odd.copy_(q)
    a, _ = m.ssm_qk_norm_rope_fwd(odd, None, w[0], None, f, pos)
    assert (a.float() - qo.float()).abs().max() <= 2.0 ** -7 * qo.float().abs().max()
    # heads in the outer dim
    a, _ = m.ssm_qk_norm_rope_fwd(q.transpose(0, 1).contiguous().transpose(0, 1), None, w[0], None, f, pos)
    assert torch.equal(a, qo)
    # cotangents as views, and dq in place
    gd = m.ssm_qk_norm_rope_bwd(q, k, w[0], w[1], f, pos, g[0], g[1])
    gv = torch.cat([g[0].flatten(1), g[1].flatten(1)], 1)
    g0, g1 = gv[:, :256].view(21, 4, 64), gv[:, 256:].view(21, 2, 64)
    ge = m.ssm_qk_norm_rope_bwd(q, k, w[0], w[1], f, pos, g0, g1)
    gi = m.ssm_qk_norm_rope_bwd(q, k, w[0], w[1], f, pos, g[0], g[1], out={"dq": g[0], "dk": g[1]})
    for n in gd:
        assert torch.equal(gd[n], ge[n]) and torch.equal(gd[n], gi[n])


def test_no_tokens(cuda_device):
    import torch
    m = lib()
    z = torch.zeros((0, 2, 64), device=cuda_device)
    w, f, pos = torch.ones(64, device=cuda_device), torch.ones(32, device=cuda_device), torch.zeros(0, dtype=torch.int32, device=cuda_device)
    a, b = m.ssm_qk_norm_rope_fwd(z, z, w, w, f, pos)
    assert a.shape == b.shape == (0, 2, 64)
    got = m.ssm_qk_norm_rope_bwd(z, z, w, w, f, pos, z, z)
    assert (got["dwq"] == 0).all() and (got["dwk"] == 0).all()


CACHES = [  # T, H, Hk, d, rot, dtype, interleaved, norm | cache, page, layout
    ((1, 4, 2, 128, 128, "bf16", False, True), "bf16", 16, "nhd"),
    ((64, 8, 2, 128, 128, "bf16", False, True), "bf16", 16, "hnd"),
    ((77, 4, 4, 72, 24, "bf16", True, True), "bf16", 1, "nhd"),
    ((130, 8, 1, 128, 64, "bf16", False, True), "f8", 64, "hnd"),
    ((50, 3, 3, 96, 48, "bf16", False, False), "f8", 24, "nhd"),
    ((45, 2, 2, 20, 8, "bf16", False, True), "f8", 8, "nhd"),
    ((90, 6, 3, 80, 40, "f32", False, True), "f32", 8, "hnd"),
    ((19, 2, 1, 33, 10, "f32", True, True), "f32", 5, "nhd"),
]


@pytest.mark.parametrize("case", CACHES, ids=lambda c: str(c) if isinstance(c, str) else None)
def test_cache(cuda_device, case):
    import torch
    shape, cache, ps, layout = case
    T, H, Hk, d, rot, dtype, il, norm = shape
    q, k, v, w, f, pos, _, flags = _make(shape, cuda_device, 7)
    rng = np.random.default_rng(8)
    pages = -(-T // ps) + 3
    slots = rng.permutation(pages * ps)[:T].astype(np.int64)
    if T > 4:
        slots[1], slots[2], slots[4] = -1, pages * ps, 1 << 40      # written nowhere
    dt = {"bf16": torch.bfloat16, "f8": torch.float8_e4m3fn, "f32": torch.float32}[cache]
    size = (pages, ps, Hk, d) if layout == "nhd" else (pages, Hk, ps, d)
    fill = torch.full(size, 3.0, device=cuda_device).to(dt)
    kc, vc = (c if layout == "nhd" else c.permute(0, 2, 1, 3) for c in (fill.clone(), fill.clone()))
    ks, vs = (0.03, 0.07) if cache == "f8" else (1.0, 1.0)
    qo = lib().ssm_qk_norm_rope_cache_fwd(q, k, v, w[0], w[1], f, pos, torch.tensor(slots, device=cuda_device), kc, vc,
                                          k_scale=ks, v_scale=vs, flags=flags)
    q2, _ = lib().ssm_qk_norm_rope_fwd(q, k, w[0], w[1], f, pos, flags=flags)
    assert torch.equal(qo, q2)
    got_k, got_v = _n(kc.float()), _n(vc.float())
    kept = (slots >= 0) & (slots < pages * ps)
    page, at = slots[kept] // ps, slots[kept] % ps
    other = np.ones((pages, ps), bool)
    other[page, at] = False
    assert (got_k[other] == 3.0).all() and (got_v[other] == 3.0).all()
    want_k = paged.qk_norm_rope(_n(k), _n(w[1]), _n(f), _n(pos), interleaved=il)[kept]
    flat = _pair(paged.qk_norm_rope(_n(k), _n(w[1]), _n(f), 0 * _n(pos), interleaved=il), rot, il)[kept]
    for n, got, want, tol, s in (("k", got_k[page, at], want_k, K * flat, ks), ("v", got_v[page, at], _n(v)[kept], 0.0, vs)):
        if cache == "f8":
            want, tol = np.clip(want / s, -448, 448), tol / s + U * np.abs(want / s)
            tol = tol + np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10)
        elif cache == "bf16" and n == "k":
            tol = tol + 2.0 ** -8 * np.abs(want)
        err = np.abs(got - want) - tol
        assert err.max() <= 0, (n, float(err.max()))


def test_cache_of_8_bits_clamps_and_keeps_nan(cuda_device):
    import torch
    m = lib()
    v = torch.tensor([0.0, 1.0, 447.0, 460.0, 1e30, float("inf"), -1e30, float("nan"), -460.0, 2.0 ** -9, 2.0 ** -11, -0.0,
                      17.0, 18.0, 19.0, 240.0], device=cuda_device).to(torch.bfloat16).view(1, 1, 16)
    kc, vc = (torch.zeros((1, 1, 1, 16), dtype=torch.uint8, device=cuda_device).view(torch.float8_e4m3fn) for _ in range(2))
    one = lambda n, t: torch.zeros(n, dtype=t, device=cuda_device)  # noqa: E731
    m.ssm_qk_norm_rope_cache_fwd(v, v, v, None, None, one(0, torch.float32), one(1, torch.int32), one(1, torch.int64), kc, vc,
                                 flags=m.SSM_QK_NO_NORM)
    want = v.float().clamp(-448, 448).to(torch.float8_e4m3fn)
    for c in (kc, vc):
        a, b = c.float().view(-1), want.float().view(-1)
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))


def test_on_a_stream_and_in_a_graph(cuda_device):
    """Captured once, replayed several times with new inputs in place, against eager calls."""
    import torch
    case = (33, 4, 2, 128, 128, "bf16", False, True)
    q, k, v, w, f, pos, g, flags = _make(case, cuda_device, 9)
    m = lib()
    outs = [torch.empty((33, n, 128), dtype=torch.bfloat16, device=cuda_device) for n in (4, 2)]
    out = {"dq": torch.empty_like(outs[0]), "dk": torch.empty_like(outs[1]),
           "dwq": torch.empty(128, device=cuda_device), "dwk": torch.empty(128, device=cuda_device)}
    ws = torch.empty(m.ssm_qk_norm_rope_bwd_workspace_size(33, 4, 2, 128), dtype=torch.uint8, device=cuda_device)

    def both():
        m.ssm_qk_norm_rope_fwd(q, k, w[0], w[1], f, pos, q_out=outs[0], k_out=outs[1])
        m.ssm_qk_norm_rope_bwd(q, k, w[0], w[1], f, pos, g[0], g[1], out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for i in range(4):
        q.copy_(torch.randn_like(q))
        pos.add_(i)
        graph.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in outs + [out[n] for n in ("dq", "dk", "dwq", "dwk")]]
        both()
        torch.cuda.synchronize()
        for a, b in zip(have, outs + [out[n] for n in ("dq", "dk", "dwq", "dwk")]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,d,dtype,both", [(4_200_003, 256, "f32", False), (1_100_001, 255, "f32", True), (8_400_001, 256, "bf16", False)])
def test_dw_of_millions_of_tokens(cuda_device, T, d, dtype, both):
    """Every token alike (one row, expanded), not rotated: dw is T times one token's term, and fp32 additions of one
    term, each rounded the same way for long, drift with their number.  A lane adds up hundreds of terms here.
    Of those at most 32 in a row are fp32, then 6 of lane groups and 8 of waves, and a few roundings to and
    from fp64: 50 u.  With x = 1 and eps = 0 a term is its cotangent itself; else it is within 40 u of itself."""
    import torch
    rng = np.random.default_rng(41)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    t = lambda a: torch.tensor(np.asarray(a, np.float32), device=cuda_device).to(dt)  # noqa: E731
    x = t(np.ones((1, 1, d)) if dtype == "f32" else rng.standard_normal((1, 1, d)))
    dy = t(rng.standard_normal((1, 1, d)))
    w = torch.ones(d, device=cuda_device)
    pos = torch.zeros(1, dtype=torch.int32, device=cuda_device).expand(T).contiguous()
    xs, gs = x.expand(T, 1, d), dy.expand(T, 1, d)
    out = {"dq": torch.empty((T, 1, d), dtype=dt, device=cuda_device)}
    if both:
        out["dk"] = torch.empty_like(out["dq"])
    eps = 0.0 if dtype == "f32" else 1e-6
    got = lib().ssm_qk_norm_rope_bwd(xs, xs if both else None, w, w if both else None, torch.zeros(0, device=cuda_device), pos, gs,
                                     gs if both else None, eps=eps, out=out)
    term = _n(dy)[0, 0] * _n(x)[0, 0] / np.sqrt((_n(x) ** 2).mean() + eps)
    for n in ("dwq", "dwk") if both else ("dwq",):
        _check("rope %s of %d tokens" % (n, T), got[n], T * term, (50 + (40 if dtype == "bf16" else 0)) * U * T * np.abs(term))


def test_in_place_where_a_dim_has_one_entry(cuda_device):
    """Contiguous as torch counts it: the stride of a token or a head that is alone means nothing."""
    import torch
    m = lib()
    gen = torch.Generator(device=cuda_device).manual_seed(51)
    r = lambda *s: torch.randn(s, generator=gen, device=cuda_device).to(torch.bfloat16)  # noqa: E731
    w, f = torch.rand(64, device=cuda_device) + 0.5, torch.rand(32, device=cuda_device)
    for T, H, Hk in ((1, 4, 2), (9, 1, 1), (1, 1, 1)):
        pos = torch.arange(T, dtype=torch.int32, device=cuda_device)
        make = (lambda h: r(1, 7, 64)[:, :h]) if T == 1 else (lambda h: r(T, 64).as_strided((T, 1, 64), (64, 1000, 1)))
        q, k, gq, gk = make(H), make(Hk), make(H), make(Hk)
        assert q.is_contiguous() and (q.stride(0) != H * 64 or q.stride(1) != 64)
        want = m.ssm_qk_norm_rope_fwd(q, k, w, w, f, pos)
        grads = m.ssm_qk_norm_rope_bwd(q, k, w, w, f, pos, gq, gk)
        got = m.ssm_qk_norm_rope_bwd(q, k, w, w, f, pos, gq, gk, out={"dq": gq, "dk": gk})
        assert got["dq"].data_ptr() == gq.data_ptr() and all(torch.equal(got[n], grads[n]) for n in grads)
        cache = [torch.zeros((1, 16, Hk, 64), dtype=torch.bfloat16, device=cuda_device) for _ in range(2)]
        qc = q.clone()
        assert qc.stride() == q.stride()
        a = m.ssm_qk_norm_rope_cache_fwd(qc, k, k, w, w, f, pos, pos.long(), *cache, q_out=qc)
        assert a.data_ptr() == qc.data_ptr() and torch.equal(a, want[0])
        a, b = m.ssm_qk_norm_rope_fwd(q, k, w, w, f, pos, q_out=q, k_out=k)
        assert a.data_ptr() == q.data_ptr() and torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("il", [False, True])
def test_far_and_negative_positions(cuda_device, il):
    """Positions up to the ends of 32 bits.  Formed and reduced in fp64, an angle there is off by up to 2^-53 of
    the product's three roundings each: 3 * 2^-53 * 2^31 = 12 u, beside the 32 u of the rest."""
    import torch
    T, H, d = 64, 2, 64
    rng = np.random.default_rng(61)
    q = torch.tensor(rng.standard_normal((T, H, d)), dtype=torch.float32, device=cuda_device)
    w = torch.tensor(rng.normal(1, 0.1, d), dtype=torch.float32, device=cuda_device)
    f = torch.tensor(1e4 ** (-np.arange(d // 2) / (d // 2)), dtype=torch.float32, device=cuda_device)
    at = np.concatenate([2 ** 31 - 1 - np.arange(24), -2 ** 31 + np.arange(16), -np.arange(12), 2 ** np.arange(12, 24)])
    pos = torch.tensor(at, dtype=torch.int32, device=cuda_device)
    m = lib()
    y, _ = m.ssm_qk_norm_rope_fwd(q, None, w, None, f, pos, flags=m.SSM_ROPE_INTERLEAVED if il else 0)
    # the angle's whole turns taken off in more than 64 bits before the oracle's cosines
    turn = np.longdouble(2) * np.arctan2(np.longdouble(0), np.longdouble(-1))
    th = np.asarray(at, np.longdouble)[:, None] * _n(f).astype(np.longdouble)[None]
    th = (th - turn * np.rint(th / turn)).astype(np.float64)[:, None]
    flat = paged.qk_norm_rope(_n(q), _n(w), _n(f), 0 * _n(pos), interleaved=il)
    a, b = (slice(0, d, 2), slice(1, d, 2)) if il else (slice(0, d // 2), slice(d // 2, d))
    want = flat.copy()
    want[..., a] = flat[..., a] * np.cos(th) - flat[..., b] * np.sin(th)
    want[..., b] = flat[..., b] * np.cos(th) + flat[..., a] * np.sin(th)
    _check("rope far positions %d" % il, y, want, (32 + 12) * U * _pair(flat.copy(), d, il))


def test_backward_of_lanes_with_many_heads(cuda_device):
    """More than 32 heads a lane with tokens that differ, turned (one element a lane): bounds as of the other shapes,
    and twice the same; and of tokens alike (vectors of four) every row of dq the same and within its bound."""
    import torch
    case = (80000, 6, 3, 31, 10, "bf16", False, True)
    test_backward(cuda_device, case)
    q, k, v, w, f, pos, g, flags = _make(case, cuda_device, 2)
    a, b = (lib().ssm_qk_norm_rope_bwd(q, k, w[0], w[1], f, pos, g[0], g[1]) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)

    q, k, v, w, f, pos, g, flags = _make((1, 1, 1, 64, 32, "f32", True, True), cuda_device, 3)
    T = 1_000_000
    row = lambda t: t.expand(T, -1, -1)  # noqa: E731
    got = lib().ssm_qk_norm_rope_bwd(row(q), row(k), w[0], w[1], f, pos.expand(T).contiguous(), row(g[0]), row(g[1]), flags=flags)
    for n, x, wx, gx in (("q", q, w[0], g[0]), ("k", k, w[1], g[1])):
        dx, _ = paged.qk_norm_rope_bwd(_n(x), _n(wx), _n(f), _n(pos), _n(gx), interleaved=True)
        size = _pair(np.abs(_n(gx)), 32, True)
        r = 1.0 / np.sqrt((_n(x) ** 2).mean(-1, keepdims=True) + 1e-6)
        wg, nx = np.abs(_n(wx)) * size, np.abs(_n(x)) * r
        assert (got["d" + n] == got["d" + n][:1]).all()
        _check("rope alike d" + n, got["d" + n][:1], dx, 64 * U * r * (wg + nx * (wg * nx).mean(-1, keepdims=True)))
