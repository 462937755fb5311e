"""Results of the long-context operators that a NaN cannot pass: every o, lse and mass is compared by a ratio that is
infinite where the result is not a number, with workspaces that hold NaN before the call; and mass is moved bit for bit.
Bounds as in longctx_cases.attention_bound and test_kv_evict_gpu.py."""
import numpy as np
import pytest
import torch

from helpers import lib, report
from longctx_cases import EDGES, U, Paged, attended, n64, ratios
from oracle import longctx
from test_kv_evict_gpu import GROWN, MASS, Step
from test_longctx_ranges_gpu import MANY, _wide
from test_page_select_gpu import ATTN, _lists
from test_prefix_attn_gpu import CASES, Shared

pytestmark = pytest.mark.gpu


def _nan(size, device):
    return torch.full((max(size, 1),), 255, dtype=torch.uint8, device=device)


def _finite(name, got, want, rows_of, q, sc, bf):
    ro, rl = ratios(got, want, rows_of, q, sc, bf, 0.0)
    report(name, o_of_bound=float(ro.max()), lse_of_bound=float(rl.max()))
    assert (ro <= 1.0).all() and (rl <= 1.0).all()


# one row whose own tokens are cut into pieces, and some of each list
ALONE = [([129], [0], [3000], 8, 2, 128, "bf16", 16, "nhd"), ([2000], [0], [3000], 4, 1, 64, "f8", 16, "hnd"), ([33], [0], [3000], 4, 2, 128, "f32", 16, "nhd"),
         ([500], [-1], [5000], 8, 8, 256, "bf16", 16, "nhd"), ([500], [0], [0], 4, 2, 256, "f32", 16, "nhd")]
PREFIX = [(c, False) for c in ALONE + CASES[:6] + CASES[7:9] + CASES[10:22] + CASES[24:]] + [(c, True) for c in MANY]


@pytest.mark.parametrize("case,room", PREFIX, ids=lambda c: "room%d" % c if isinstance(c, bool) else "%d-%d-%d-H%d-%d-d%d-%s-p%d-%s" % ((max(c[0]), len(c[0]), max(c[2])) + c[3:]))
def test_prefix_attention(cuda_device, case, room):
    s = Shared(cuda_device, 170 + case[5], *case)
    if room:
        _wide(s)
    ws = _nan(lib().ssm_prefix_attn_decode_fwd_workspace_size(len(s.rows), s.H, s.Hk, s.d, s.ptable.shape[1], s.own.shape[1], s.ps), cuda_device)
    _finite("finite prefix %s" % (case[3:],), s.call(workspace=ws), s.want(), attended(s), s.q, s.sc, s.cache != "f32")


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "%d-%d-H%d-%d-d%d-%s-p%d-%s-k%d" % ((len(c[0]), max(c[0])) + c[1:]))
def test_attention_over_chosen_pages(cuda_device, case):
    lens, H, Hk, d, cache, ps, layout, top_k = case
    c = Paged(cuda_device, 180 + d, lens, Hk, d, cache, ps, layout)
    q, sc = c.queries(len(lens), H, d), d ** -0.5
    sel = _lists(c.rng, lens, c.table, Hk, ps, top_k)
    ws = _nan(lib().ssm_select_attn_decode_fwd_workspace_size(len(lens), H, Hk, d, c.table.shape[1], ps, top_k), cuda_device)
    got = lib().ssm_select_attn_decode_fwd(q, c.k, c.v, c.t(c.table), c.t(lens), c.t(sel), scale=sc, k_scale=c.scale, v_scale=c.scale, return_lse=True,
                                           workspace=ws)
    k64, v64 = c.k64(), c.v64()
    want = longctx.select_attn_decode(n64(q), k64, v64, c.table, lens, sel, sc)
    tokens = [longctx._tokens(c.table[r], lens[r], ps, c.pages) for r in range(len(lens))]

    def rows_of(r, h):
        g = h * Hk // H
        held = -(-min(max(int(lens[r]), 0), c.table.shape[1] * ps) // ps)
        at = [t for i in sel[r][g][:held] for t in tokens[r][int(i) * ps:(int(i) + 1) * ps] if i >= 0]
        p, i = [t[1] for t in at], [t[2] for t in at]
        return k64[p, i, g].reshape(-1, d), v64[p, i, g].reshape(-1, d)

    _finite("finite chosen %s" % (case[1:],), got, want, rows_of, q, sc, cache != "f32")


@pytest.mark.parametrize("case", MASS + [([0] * 20, EDGES, 8, 1, 128, "bf16", 16, "nhd"), (GROWN, EDGES, 32, 1, 256, "f32", 16, "nhd")],
                         ids=lambda c: "%d-%d-H%d-%d-d%d-%s-p%d-%s" % ((len(c[0]), max(c[1])) + c[2:]))
def test_gathered_weight(cuda_device, case):
    """mass holds NaN wherever no token from before has weight."""
    s = Step(cuda_device, 190 + case[4], *case)
    held = np.zeros((s.pages, s.ps), bool)
    for r in range(len(s.lens)):
        for j, p, i in longctx._tokens(s.table[r], min(s.old[r], s.lens[r]), s.ps, s.pages):
            held[p, i] = True
    s.mass.masked_fill_(torch.tensor(~held, device=cuda_device)[:, None, :], float("nan"))
    was, k64, q64, lse = n64(s.mass), s.k64(), n64(s.q), n64(s.lse)
    want = longctx.mass_update(q64, k64, lse, was, s.table, s.starts, s.pos, s.old, s.lens, s.sc)
    s.call()
    got, worst = n64(s.mass), 0.0
    touched = np.zeros(got.shape, bool)
    for r in range(len(s.lens)):
        at = longctx._tokens(s.table[r], s.lens[r], s.ps, s.pages)
        if not at:
            continue
        p, i = np.array([t[1] for t in at]), np.array([t[2] for t in at])
        touched[p, :, i] = True
        a, b = s.starts[r], s.starts[r + 1]
        # of the request's largest products, lse and rows: what each token's own are at most
        x = abs(s.sc) * (np.abs(q64[a:b]).reshape(-1, s.d) @ np.abs(k64[p, i]).reshape(-1, s.d).T).max(initial=0.0) if b > a else 0.0
        low = np.abs(lse[a:b][np.isfinite(lse[a:b])]).max(initial=0.0)
        each = (s.d + 6) * U * x + 2 * U * (x + low) + 2 * U
        w = want[p, :, i]
        tol = w * (1.5 * each + ((b - a) * s.H / s.Hk / 16 + 8) * U) + U * w + 1e-37
        ratio = np.abs(got[p, :, i] - w) / tol
        worst = max(worst, float(np.where(np.isnan(ratio), np.inf, ratio).max()))
    np.testing.assert_array_equal(got[~touched], was[~touched])
    report("finite mass %s" % (case[2:],), of_bound=worst)
    assert worst <= 1.0


@pytest.mark.parametrize("case", [([1000, 2100, 902, 0, 7], 2, 16, 16, 333, 32), ([3000, 5], 1, 64, 16, 2999, 0), ([400] * 9, 3, 5, 5, 64, 64)],
                         ids=lambda c: "%d-Hk%d-p%d-b%d-%d" % (max(c[0]), c[1], c[3], c[4], c[5]))
def test_mass_moves_bit_for_bit(cuda_device, case):
    """NaN of any payload and zeros of either sign among the mass: the kept ones are where they should be, as the bits they
    were, and everything else is untouched."""
    lens, Hk, d, ps, budget, recent = case
    c = Paged(cuda_device, 200, lens, Hk, 16, "bf16", ps, nan=False)
    bits = np.exp(c.rng.standard_normal((c.pages, Hk, ps))).astype(np.float32).view(np.int32)
    strange = np.array([0x7fc00001, 0x7f800001, -1, 0x7fabcdef, 0, -(1 << 31), 0x7f800000, 1, -0x7fffffff, -0x00800000], np.int32)
    bits = np.where(c.rng.random(bits.shape) < 0.2, c.rng.choice(strange, bits.shape), bits)
    mass = torch.tensor(bits, device=cuda_device).view(torch.float32)
    _, _, _, length, kept = longctx.evict(np.zeros((c.pages, ps, Hk, 1)), np.zeros((c.pages, ps, Hk, 1)), bits.view(np.float32), c.table, lens, budget, recent)
    n, got = lib().ssm_kv_evict(c.k, c.v, mass, c.t(c.table), c.t(lens), budget=budget, recent=recent)
    np.testing.assert_array_equal(n.cpu().numpy(), length)
    np.testing.assert_array_equal(got.cpu().numpy(), kept)
    want = bits.copy()
    for r, m in enumerate(lens):
        for g in range(Hk if m > budget else 0):
            i, j = np.arange(budget), kept[r, g]
            want[c.table[r, i // ps], g, i % ps] = bits[c.table[r, j // ps], g, j % ps]
    np.testing.assert_array_equal(mass.view(torch.int32).cpu().numpy(), want)
