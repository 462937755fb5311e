"""ssm_prefix_attn_decode_fwd where V is not finite: what a prefix holds reaches the rows behind it and no others, whatever
rows stand next to each other.  Bounds as in test_prefix_attn_gpu.py."""
import numpy as np
import pytest

from helpers import report
from longctx_cases import n64, ratios
from oracle import longctx
from test_longctx_ranges_gpu import _wide
from test_prefix_attn_gpu import Shared

pytestmark = pytest.mark.gpu

LENS = [5, 0, 17, 3, 1, 0, 64, 2]
THREE, TWO = [100, 200, 300], [100, 20]
# Prefix lengths, prefix of each row, own lengths, H, Hk, d, cache, page, layout; room for long prefixes (with many columns:
# the form for many).  So many rows or kv heads that a block has the whole of its rows' prefixes, except in the last of
# each form, where parts end in the middle of one.
MIXED = [
    # up to 16 columns of a kv head
    ((THREE, [0, 1, 2, -1, 0, 2, 1, 9], LENS, 512, 256, 64, "bf16", 16, "nhd"), False),
    ((TWO, [0, 1, 0, -1, 0, 1, 1, 0], LENS, 256, 256, 256, "bf16", 16, "hnd"), False),
    ((TWO, [0, 1, 0, -1, 0, 1, 1, 0], LENS, 256, 256, 128, "f8", 16, "nhd"), False),
    ((TWO, [1, 0, 0, -1, 0, 1, 1, 0], LENS, 256, 256, 72, "f32", 16, "nhd"), False),
    # up to 32 of a block
    ((THREE, [0, 1, 2, -1] * 18, LENS * 9, 16, 1, 128, "bf16", 16, "hnd"), False),
    ((THREE, [0, 1, 2, -1] * 51, [1, 0, 2, 3] * 51, 5, 1, 96, "bf16", 24, "nhd"), False),
    ((TWO, [0, 1, -1, 0] * 2, LENS, 768, 256, 256, "bf16", 16, "nhd"), False),
    ((THREE, [2, 1, 0, -1] * 18, LENS * 9, 16, 1, 64, "f8", 64, "hnd"), False),
    ((TWO, [0, 1, -1, 0] * 2, LENS, 768, 256, 192, "f8", 16, "nhd"), False),
    ((THREE, [0, 1, 2, -1] * 18, LENS * 9, 16, 1, 128, "f32", 16, "nhd"), False),
    ((TWO, [0, 1, -1, 0] * 2, LENS, 768, 256, 256, "f32", 16, "nhd"), False),
    ((TWO, [0, 1, 0, -1, 0, 1, 1, 0], LENS, 4, 2, 256, "f32", 16, "hnd"), False),
    # many
    ((THREE, [0, 1, 2, -1] * 130, [1, 0, 2, 3] * 130, 16, 1, 128, "bf16", 16, "nhd"), True),
    ((THREE, [0] * 173 + [1] * 173 + [2] * 174, [1, 0, 2, 3] * 130, 16, 1, 80, "bf16", 16, "hnd"), True),
    ((THREE, [2, 1, 0, -1] * 130, [1, 0, 2, 3] * 130, 16, 1, 64, "f8", 64, "hnd"), True),
    ((THREE, [0, 1, 2, -1] * 130, [1, 0, 2, 3] * 130, 16, 1, 64, "f32", 16, "nhd"), True),
    ((THREE, [0, 1, 2, -1] * 130, [1, 0, 2, 3] * 130, 16, 1, 128, "f32", 16, "nhd"), True),
    ((THREE, [0, 1, 2, -1] * 33, [1, 0, 2, 3] * 33, 16, 1, 256, "bf16", 16, "nhd"), False),
    ((THREE, [1, 2, 0, -1] * 33, [1, 0, 2, 3] * 33, 16, 1, 256, "f8", 16, "hnd"), False),
    ((THREE, [0, 1, 2, -1] * 33, [1, 0, 2, 3] * 33, 16, 1, 192, "f32", 16, "nhd"), False),
    (([100, 1500, 970], [0, 1, 2, -1] * 66, [1, 0, 2, 3] * 66, 16, 1, 64, "bf16", 16, "nhd"), True),
]


@pytest.mark.parametrize("case,many", MIXED, ids=lambda c: c if isinstance(c, bool) else "%d-H%d-%d-d%d-%s-p%d-%s" % ((len(c[2]),) + c[3:]))
def test_values_that_are_not_finite_reach_their_own_rows_alone(cuda_device, case, many):
    """NaN and infinities in V of tokens of the first prefix, and of one row's own token."""
    s = Shared(cuda_device, 160 + case[5], *case)
    if many:
        _wide(s)
    v0 = s.v64()
    bad = [float("nan")] * 3 if case[6] == "f8" else [float("inf"), -float("inf"), float("nan")]
    dims = (1, case[5] // 2, case[5] - 3)
    for j, x, dim in zip((0, 41, 99), bad, dims):
        s.v[int(s.ptable[0, j // s.ps]), j % s.ps, :, dim] = x
    s.v[int(s.own[2, 0]), 0, :, 0] = float("nan")
    got = s.call()

    def tokens(r):
        p = s.prefix[r]
        t = longctx._tokens(s.ptable[p], s.plens[p], s.ps, s.pages) if 0 <= p < len(s.plens) else []
        t = t + longctx._tokens(s.own[r], s.rows[r], s.ps, s.pages)
        return np.array([x[1] for x in t], int), np.array([x[2] for x in t], int)

    at, k64 = [tokens(r) for r in range(len(s.rows))], s.k64()
    want = longctx.prefix_attn_decode(n64(s.q), k64, v0, s.prefix, s.ptable, s.plens, s.own, s.rows, s.sc)
    bf = s.cache != "f32"
    ro, rl = ratios(got, want, lambda r, h: (k64[(*at[r], h * s.Hk // s.H)], v0[(*at[r], h * s.Hk // s.H)]), s.q, s.sc, bf,
                    2.0 ** -17 if bf else 0.0)
    hit = np.zeros(ro.shape, bool)
    for dim in dims:
        hit[s.prefix == 0, :, dim] = True
    hit[2, :, 0] = True
    report("values %s" % (case[3:],), o_of_bound=float(ro[~hit].max()), lse_of_bound=float(rl.max()))
    assert np.isinf(ro[hit]).all()
    assert (ro[~hit] <= 1.0).all() and (rl <= 1.0).all(), np.argwhere((ro > 1.0) & ~hit)[:5]
