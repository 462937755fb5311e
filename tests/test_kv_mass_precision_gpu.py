"""How many bits ssm_kv_mass_update keeps of a large lse: scores of several hundred that are exact, so that nothing but lse
itself could move the weights."""
import numpy as np
import pytest
import torch

from helpers import lib, report
from longctx_cases import U, Paged, n64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "f8", "f32"])
@pytest.mark.parametrize("rows", [1, 150])
@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_weights_of_a_large_lse(cuda_device, rows, d, cache):
    """Request r's queries have the score S_r with each of its tokens, a scale of ln 2, so log2(e) scale is 1 in fp32: the
    exponent S_r - log2(e) lse is exact where log2(e) lse is not rounded, and each weight exp(S_r scale - lse) of some 1/200 is off by
    |S_r| |1 - log2(e) scale| (the scale's own rounding, 2^-28 or so of S_r), two powers of two of 2 u each, and for a sum of n weights
    (n / 16 + 8) u more.  A rounded log2(e) lse would move all weights of a request by up to u |S_r| of themselves, 300 u and more."""
    S = np.array([257, 301, 333, 421, 499, 555, 601, 677, 743, 801, 847, 911, 953, 999, 1001, -267, -555, -1003, 1023, 2047], float)
    S = torch.tensor(S).to(torch.bfloat16).double().numpy()
    n = np.array([200 + 3 * i for i in range(len(S))])
    c = Paged(cuda_device, 90, n, 1, d, cache, 16)
    k = torch.full(c.k.shape, float("nan"), device=cuda_device)
    used = torch.tensor(c.used(), device=cuda_device)
    k[used] = 0.0
    k[..., 0][used] = 1.0 / c.scale
    c.k = k.to(c.k.dtype)
    sc = float(np.float32(np.log(2.0)))
    assert np.float32(sc) * np.float32(1.4426950408889634) == 1.0
    q = torch.zeros((len(S) * rows, 1, d), device=cuda_device)
    q[:, 0, 0] = torch.tensor(np.repeat(S, rows), device=cuda_device)
    lse = np.repeat(S * sc + np.log(n), rows).astype(np.float32)
    pos = np.concatenate([np.arange(m - rows, m) for m in n])
    mass = torch.full((c.pages, 1, 16), float("nan"), device=cuda_device)
    lib().ssm_kv_mass_update(q.to(torch.float32 if cache == "f32" else torch.bfloat16), c.k, torch.tensor(lse, device=cuda_device)[:, None], mass, c.t(c.table),
                             c.t(np.arange(len(S) + 1) * rows), c.t(pos), c.t(np.zeros(len(S))), c.t(n), scale=sc, k_scale=c.scale)
    got, worst = n64(mass), 0.0
    for r, m in enumerate(n):
        j = np.arange(m)
        see = np.minimum(m - j, rows)
        want = see * np.exp(S[r] * sc - float(lse[r * rows]))
        tol = want * (abs(S[r] * (1 - sc / np.log(2.0))) + (4 + see / 16 + 8) * U)
        worst = max(worst, float((np.abs(got[c.table[r, j // 16], 0, j % 16] - want) / tol).max()))
        assert np.isfinite(worst)
    report("mass of a large lse %d rows d %d %s" % (rows, d, cache), of_bound=worst)
    assert worst <= 1.0, worst
