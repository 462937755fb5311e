"""CPU pins of the fp64 oracle of the paged-attention operators (oracle/paged.py):

  * pages: a hand case; pages are never lost or held twice over many random steps, and
    every slot lies on a page that its request holds;
  * norm and rotation: the rotation as complex turns, the inner product of two rotated
    heads depends on the distance alone, unit mean square of a normed head; its gradients
    against central differences and the adjoint identity;
  * attention: against a materialised softmax over gathered rows, the mean of v at q = 0,
    one token, a window, rows without tokens and without valid pages.
"""
import numpy as np
import pytest

from oracle import paged


def test_pages_hand_case():
    # 2 tokens a page; ring of 6 starts at place 4: free pages 7, 8, 9 (wrapping)
    table = np.array([[1, -1, -1], [2, 3, -1], [4, -1, -1], [5, -1, -1]])
    ring = np.array([9, -1, -1, -1, 7, 8])
    got = paged.pages_step([2, 3, 1, 2], [4, 0, 2, 9], table, ring, [4, 3], 2, 6)
    assert got["block_table"].tolist() == [[1, 7, -1], [2, 3, -1], [4, -1, -1], [5, -1, -1]]
    assert got["free_ring"].tolist() == [9, 2, 3, -1, 7, 8]     # 2 and 3 given back behind 9
    assert got["ring"].tolist() == [5, 4]
    assert got["len"].tolist() == [4, 0, 2, 2] and got["denied"].tolist() == [1]   # 9 tokens: 5 pages > 3
    assert got["starts"].tolist() == [0, 2, 2, 3, 10]
    assert got["request"].tolist() == [0, 0, 2, 3, 3, 3]
    assert got["positions"].tolist() == [2, 3, 1, 2, 3, 4]
    assert got["slots"].tolist() == [14, 15, 9, -1, -1, -1]


@pytest.mark.parametrize("ps", [1, 3, 16])
def test_pages_are_kept(ps):
    rng = np.random.default_rng(ps)
    n, cols, batch = 40, 9, 7
    ring, place = [3, n], rng.permutation(n)
    table, held = np.full((batch, cols), -1), np.zeros(batch, int)
    for _ in range(60):
        new = np.where(rng.random(batch) < 0.3, 0, held + rng.integers(0, 3 * ps, batch))
        got = paged.pages_step(held, new, table, place, ring, ps, 200)
        table, place, ring, held = got["block_table"], got["free_ring"], got["ring"], got["len"]
        pages = [int(p) for r in range(batch) for p in table[r, :-(-held[r] // ps)]]
        pages += [int(place[(ring[0] + i) % n]) for i in range(ring[1])]
        assert sorted(pages) == list(range(n))
        for t in np.flatnonzero(got["slots"] >= 0):
            r, p = got["request"][t], got["positions"][t]
            assert got["slots"][t] == table[r, p // ps] * ps + p % ps
        assert (held <= cols * ps).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_as_complex_turns(interleaved, norm):
    rng = np.random.default_rng(3)
    T, H, d, rot = 5, 3, 10, 6
    x, w = rng.standard_normal((T, H, d)), rng.normal(1, 0.1, d)
    f, pos = rng.random(rot // 2), np.array([0, 1, 7, 100000, -2])
    y = paged.qk_norm_rope(x, w if norm else None, f, pos, interleaved=interleaved)
    z = x * w / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) if norm else x
    a, b = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(rot // 2), np.arange(rot // 2, rot))
    c = (z[..., a] + 1j * z[..., b]) * np.exp(1j * pos[:, None, None] * f)
    np.testing.assert_allclose(y[..., a] + 1j * y[..., b], c, rtol=1e-9, atol=1e-9)
    np.testing.assert_array_equal(y[..., rot:], z[..., rot:])


def test_rope_products_depend_on_distance():
    rng = np.random.default_rng(4)
    x, f = rng.standard_normal((2, 1, 8)), rng.random(4)
    prods = []
    for p in (0, 11, 900):
        y = paged.qk_norm_rope(x, None, f, [p + 5, p])
        prods.append(float(y[0, 0] @ y[1, 0]))
    np.testing.assert_allclose(prods, prods[0], rtol=1e-10)
    y = paged.qk_norm_rope(rng.standard_normal((3, 2, 16)), np.ones(16), f, [1, 2, 3], eps=0.0)
    np.testing.assert_allclose((y ** 2).mean(-1), 1.0, rtol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_bwd_against_differences(interleaved, norm):
    rng = np.random.default_rng(5)
    T, H, d, rot = 3, 2, 7, 4
    x, w, g = rng.standard_normal((T, H, d)), rng.normal(1, 0.2, d) if norm else None, rng.standard_normal((T, H, d))
    f, pos = rng.random(rot // 2), [2, 0, 31]
    fwd = lambda x, w: float((paged.qk_norm_rope(x, w, f, pos, eps=1e-3, interleaved=interleaved) * g).sum())  # noqa: E731
    dx, dw = paged.qk_norm_rope_bwd(x, w, f, pos, g, eps=1e-3, interleaved=interleaved)
    h = 1e-5
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        np.testing.assert_allclose(dx[i], (fwd(x + e, w) - fwd(x - e, w)) / (2 * h), rtol=1e-6, atol=1e-8)
    if norm:
        for i in range(d):
            e = np.zeros(d)
            e[i] = h
            np.testing.assert_allclose(dw[i], (fwd(x, w + e) - fwd(x, w - e)) / (2 * h), rtol=1e-6, atol=1e-8)
        np.testing.assert_allclose((dw * w).sum(), fwd(x, w), rtol=1e-10)     # linear in w
    else:
        assert dw is None
        np.testing.assert_allclose((dx * x).sum(), fwd(x, w), rtol=1e-10)     # linear in x


def test_attn_against_a_materialised_softmax():
    rng = np.random.default_rng(6)
    B, H, Hk, d, ps, cols, P = 4, 6, 2, 8, 3, 5, 24
    kc, vc = rng.standard_normal((P, ps, Hk, d)), rng.standard_normal((P, ps, Hk, d))
    q, table, lens = rng.standard_normal((B, H, d)), rng.permutation(P)[:B * cols].reshape(B, cols), [15, 1, 0, 7]
    for window in (0, 4):
        o, lse = paged.paged_attn_decode(q, kc, vc, table, lens, 0.3, window)
        for r in range(B):
            k, v = kc[table[r]].reshape(-1, Hk, d), vc[table[r]].reshape(-1, Hk, d)
            keep = np.arange(cols * ps) < lens[r]
            if window:
                keep &= np.arange(cols * ps) >= lens[r] - window
            for h in range(H):
                g = h // (H // Hk)
                p = np.where(keep, np.exp(0.3 * (k[:, g] @ q[r, h])), 0.0)
                if not keep.any():
                    assert (o[r, h] == 0).all() and lse[r, h] == -np.inf
                    continue
                np.testing.assert_allclose(o[r, h], p @ v[:, g] / p.sum(), rtol=1e-12)
                np.testing.assert_allclose(lse[r, h], np.log(p.sum()), rtol=1e-12)


def test_attn_limits():
    rng = np.random.default_rng(7)
    kc, vc = rng.standard_normal((3, 4, 1, 8)), rng.standard_normal((3, 4, 1, 8))
    q = rng.standard_normal((1, 2, 8))
    o, lse = paged.paged_attn_decode(0 * q, kc, vc, [[2, 0]], [6], 1.0)
    np.testing.assert_allclose(o[0, 0], np.concatenate([vc[2, :, 0], vc[0, :2, 0]]).mean(0), rtol=1e-12)
    np.testing.assert_allclose(lse, np.log(6), rtol=1e-12)
    o, lse = paged.paged_attn_decode(q, kc, vc, [[1, 0]], [1], 0.5)
    np.testing.assert_allclose(o[0], np.tile(vc[1, 0], (2, 1)), rtol=1e-12)
    np.testing.assert_allclose(lse[0], 0.5 * q[0] @ kc[1, 0, 0], rtol=1e-12)
    o, lse = paged.paged_attn_decode(q, kc, vc, [[-1, 3]], [8], 0.5)     # no valid page
    assert (o == 0).all() and (lse == -np.inf).all()
    a, _ = paged.paged_attn_decode(q, kc, vc, [[1, 7]], [8], 0.5)        # the second page is left out
    b, _ = paged.paged_attn_decode(q, kc, vc, [[1, 0]], [4], 0.5)
    np.testing.assert_array_equal(a, b)
