"""How many bits ssm_prefix_attn_decode_fwd keeps, where its inputs leave nothing else to hide behind: outputs in which the
tokens' shares nearly cancel, so that an error of a weight is far above the output's own rounding.

A prefix has two tokens, of scores 0 and s in [-1.2, 0): weights 1, exactly, and p = exp(s).  s is a sum of two products,
exact but for one rounding, times log2(e), rounded twice, so its exponential is within 4 u |s| + 2 u < 8 u of p (u = 2^-24)
where 2^x is within 2 u of itself; products with v and their sums in fp32 are at most six roundings of what they add up, and
the quotient two more: 16 u (|v0| + p |v1|) / (1 + p) in all, with the output's own rounding behind it, 2^-8 |o|.  A weight
of 17 bits is off by up to 2^-18, 64 u.  v0 = -n1, v1 = n2 and q are such that p n2 is n1 (1 + 2^-14) or so, for each (row, head)
in one dim of its own."""
import numpy as np
import pytest
import torch

from helpers import report
from longctx_cases import U, n64
from test_longctx_ranges_gpu import _wide
from test_prefix_attn_gpu import Shared

pytestmark = pytest.mark.gpu

# rows, H, Hk, d, cache; room for long prefixes (with many columns: the form for many)
FORMS = [(7, 4, 2, 64, "bf16", False), (7, 2, 2, 128, "bf16", False), (40, 8, 4, 80, "bf16", False), (3, 4, 1, 256, "bf16", False),
         (7, 4, 2, 128, "f8", False), (40, 4, 2, 96, "f8", False), (5, 4, 1, 256, "f8", False),
         (100, 16, 2, 64, "bf16", True), (100, 16, 2, 128, "bf16", True), (100, 16, 2, 72, "bf16", True), (40, 8, 1, 256, "bf16", True),
         (100, 16, 2, 64, "f8", True), (100, 16, 2, 128, "f8", True), (40, 8, 1, 192, "f8", True)]
IDS = ["%d-H%d-%d-d%d-%s-%s" % (f[:5] + ("many" if f[5] else "few",)) for f in FORMS]


class Two(Shared):
    """Rows behind one prefix of two tokens, and no tokens of their own."""

    def __init__(self, device, rows, H, Hk, d, cache, room):
        super().__init__(device, 7, [2], [0] * rows, [0] * rows, H, Hk, d, cache, 16, nan=False)
        if room:
            _wide(self)
        self.sc = 1.0
        n2 = 14 if cache == "f8" else 255
        n1 = np.random.default_rng(d).integers(n2 // 3, n2, d)
        page = int(self.ptable[0, 0])
        k, v = np.zeros((2, Hk, d)), np.zeros((2, Hk, d))
        k[1, :, 0], k[1, :, 1] = 1.0, 2.0 ** -8
        v[0], v[1] = -n1, n2
        for c, x in ((self.k, k), (self.v, v)):
            c[page, :2] = torch.tensor(x / self.scale, dtype=torch.float32).to(c.dtype).to(device)
        want = np.log(n1[np.arange(rows * H) % d] / n2) + 2.0 ** -14
        q = torch.zeros((rows * H, d))
        q[:, 0] = torch.tensor(want).to(torch.bfloat16).float()
        q[:, 1] = torch.tensor((want - q[:, 0].double().numpy()) * 2.0 ** 8)
        self.q = q.to(torch.bfloat16).view(rows, H, d).to(device)
        q = n64(self.q)
        self.p = np.exp(q[..., 0] + q[..., 1] * 2.0 ** -8)[..., None]
        self.v0, self.v1 = -n1.astype(float), float(n2)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_lse_keeps_all_its_bits(cuda_device, form):
    """lse = ln(1 + p): 8 u p / (1 + p) of p, a rounding of the sum, and 2 u of a logarithm below 0.7, each of them at most u: 8 u.
    A sum of weights of 17 bits is off by up to 64 u p / (1 + p)."""
    s = Two(cuda_device, *form)
    got, want = n64(s.call()[1]), np.log1p(s.p[..., 0])
    ratio = np.abs(got - want) / (8 * U)
    report("lse %s" % (form,), of_bound=float(ratio.max()))
    assert (ratio <= 1.0).all()


@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_weights_keep_all_their_bits(cuda_device, form):
    s = Two(cuda_device, *form)
    o = n64(s.call()[0])
    want = (s.v0 + s.p * s.v1) / (1 + s.p)
    bound = 16 * U * (np.abs(s.v0) + s.p * s.v1) / (1 + s.p) + 2.0 ** -8 * np.abs(want)
    ratio = np.abs(o - want) / bound
    report("weights %s" % (form,), of_bound=float(ratio.max()))
    assert (ratio <= 1.0).all()


# prefix tokens, own tokens of the rows, H, Hk, d, cache; room for long prefixes
JOINED = [(300, [299], 8, 2, 128, "bf16", False), (3000, [2999], 4, 1, 64, "f32", False), (2000, [2001], 8, 2, 128, "f8", False),
          (3000, [2999, 0, 3000, 17], 4, 2, 128, "f32", False), (900, [899, 901, 1, 0, 900, 17, 902], 6, 1, 96, "bf16", False),
          (40, [39, 41, 0, 40] * 20, 4, 2, 64, "f32", False), (40, [39, 41, 0, 40, 1] * 20, 16, 2, 128, "bf16", True),
          (40, [39, 41, 0, 40, 1] * 20, 16, 2, 64, "f8", True), (40, [39, 41, 0, 40, 1] * 20, 16, 2, 128, "f32", True),
          (2000, [1999, 2001] * 20, 4, 1, 256, "f32", False), (100, [99, 101, 100, 0] * 10, 4, 1, 256, "bf16", False)]


@pytest.mark.parametrize("score", [1024.0, -1000.0])
@pytest.mark.parametrize("case", JOINED, ids=lambda c: "%d-%d-%d-H%d-%d-d%d-%s-%s" % ((c[0], len(c[1]), max(c[1])) + c[2:6] + ("many" if c[6] else "few",)))
def test_prefix_and_own_tokens_weigh_the_same(cuda_device, case, score):
    """Every token of the prefix and of the rows' own has the same score, large and exact (a scale whose product with
    log2(e) is 1), so every weight is 1: of N values -1 and n values 1, o = (n - N) / (n + N) but for the roundings of 1 / (n + N),
    of its product and of the output.  A join by lse, in fp32, would take the own tokens' weight to be off by up to
    4 u |lse|, some 2^-12."""
    N, lens, H, Hk, d, cache, room = case
    s = Shared(cuda_device, 8, [N], [0] * len(lens), lens, H, Hk, d, cache, 16)
    if room:
        _wide(s)
    s.sc = float(np.float32(np.log(2.0)))
    assert np.float32(s.sc) * np.float32(1.4426950408889634) == 1.0
    used = torch.tensor(s.used(), device=cuda_device)
    prefix = torch.zeros(s.pages, dtype=torch.bool, device=cuda_device)
    prefix[torch.tensor(s.ptable[s.ptable >= 0], device=cuda_device)] = True
    k, v = (torch.full(s.k.shape, float("nan"), device=cuda_device) for _ in range(2))
    k[used] = 0.0
    k[..., 0][used] = 1.0 / s.scale
    v[used] = 1.0 / s.scale
    v[prefix] *= -1.0
    s.k, s.v = k.to(s.k.dtype), v.to(s.v.dtype)
    s.q = torch.zeros_like(s.q)
    s.q[..., 0] = score
    o, lse = (n64(x) for x in s.call())
    n = np.array(lens, float)
    want = ((n - N) / (n + N))[:, None, None]
    step = 4 * U if cache == "f32" else 2.0 ** -8 + 4 * U
    assert (np.abs(o - want) <= step * np.abs(want)).all(), np.abs(o - want).max()
    # the logarithm of a whole number, exact, and the maximum times ln 2: 2 u each, and a rounding of their sum
    want = (score * s.sc + np.log(n + N))[:, None]
    assert (np.abs(lse - want) <= 6 * U * (abs(score) + np.log(n + N)[:, None])).all(), np.abs(lse - want).max() / U / abs(score)
