"""What pins oracle/longctx.py: attention over one list of tokens against paged attention of the
joined sequence, brute force over bounds, upper bounds, sums of weights, hand cases."""
import numpy as np

from oracle import longctx, paged


def _cache(rng, P=30, ps=4, Hk=2, d=8):
    return rng.standard_normal((P, ps, Hk, d)), rng.standard_normal((P, ps, Hk, d))


def test_a_prefix_is_the_same_as_its_pages_before_the_rows_own():
    rng = np.random.default_rng(1)
    kc, vc = _cache(rng)
    pt = rng.permutation(30)[:10].reshape(2, 5)
    own = np.array([[20, 21], [22, 23], [24, 25], [26, 27]])
    q = rng.standard_normal((4, 6, 8))
    # prefixes that fill their pages: the joined table is theirs and then the row's
    o, lse = longctx.prefix_attn_decode(q, kc, vc, [0, 1, 0, 1], pt, [20, 20], own, [5, 0, 8, 1], 0.4)
    joined = np.concatenate([pt[[0, 1, 0, 1]], own], 1)
    wo, wl = paged.paged_attn_decode(q, kc, vc, joined, [25, 20, 28, 21], 0.4)
    np.testing.assert_allclose(o, wo, rtol=1e-12)
    np.testing.assert_allclose(lse, wl, rtol=1e-12)
    # no prefix, and none of either
    o, lse = longctx.prefix_attn_decode(q, kc, vc, [-1, 2, 0, 1], pt, [0, 3], own, [5, 0, 0, 0], 0.4)
    wo, wl = paged.paged_attn_decode(q, kc, vc, np.concatenate([own[:3], pt[1:2, :2]]), [5, 0, 0, 3], 0.4)
    np.testing.assert_allclose(o, wo, rtol=1e-12)
    np.testing.assert_allclose(lse, wl, rtol=1e-12)
    assert (o[1] == 0).all() and (lse[1:3] == -np.inf).all()


def test_bounds_and_scores():
    rng = np.random.default_rng(2)
    kc, _ = _cache(rng)
    table, lens = rng.permutation(30)[:12].reshape(2, 6), [23, 9]
    b = longctx.page_bounds(kc, np.full((30, 2, 2, 8), 9.0), table, [0, 0], lens)
    for r in range(2):
        for i in range(-(-lens[r] // 4)):
            k = kc[table[r, i], :min(4, lens[r] - 4 * i)]
            np.testing.assert_array_equal(b[table[r, i], :, 0], k.min(0))
            np.testing.assert_array_equal(b[table[r, i], :, 1], k.max(0))
    untouched = np.setdiff1d(np.arange(30), np.concatenate([table[0, :6], table[1, :3]]))
    assert (b[untouched] == 9.0).all()
    # in two steps the same as in one
    c = longctx.page_bounds(kc, np.full((30, 2, 2, 8), 9.0), table, [0, 0], [10, 9])
    np.testing.assert_array_equal(longctx.page_bounds(kc, c, table, [10, 9], lens), b)
    # no key's product exceeds its page's score, and one page of one key reaches it
    q = rng.standard_normal((4, 8))
    sc = longctx.page_scores(q, b, table[0], 6, [range(2), range(2, 4)])
    for i in range(6):
        for j in range(min(4, 23 - 4 * i)):
            for h in range(4):
                assert q[h] @ kc[table[0, i], j, h // 2] <= sc[h // 2, i] + 1e-6
    one = longctx.page_scores(q, longctx.page_bounds(kc, b, table, [0, 0], [1, 0]), table[0], 1, [range(2), range(2, 4)])
    np.testing.assert_allclose(one[1, 0], max(q[2] @ kc[table[0, 0], 0, 1], q[3] @ kc[table[0, 0], 0, 1]), rtol=1e-6)


def test_select():
    # one dim: the score is q * hi
    hi = [3.0, 9.0, 1.0, 9.0, 5.0, np.nan, 9.0, 2.0]
    b = np.stack([np.zeros(8), hi], -1).reshape(8, 1, 2, 1)
    t = np.arange(8)[None]
    sel = lambda n, k, first, last: longctx.page_select(np.ones((1, 1, 1)), b, t, [n], 4, k, first, last)[0, 0].tolist()  # noqa: E731
    assert sel(32, 3, 0, 0) == [1, 3, 5]              # the NaN, then the lowest of equal ones
    assert sel(32, 5, 1, 1) == [0, 1, 3, 5, 7]
    assert sel(20, 2, 0, 1) == [1, 4] and sel(17, 3, 0, 0) == [1, 3, 4]
    assert sel(8, 4, 1, 1) == [0, 1, -1, -1] and sel(0, 2, 0, 1) == [-1, -1] and sel(13, 4, 0, 0) == [0, 1, 2, 3]
    assert sel(32, 3, 3, 0) == [0, 1, 2] and sel(30, 2, 0, 2) == [6, 7]
    t[0, 1] = 99                                      # not in the cache
    assert sel(32, 3, 0, 0) == [3, 5, 6]


def test_select_attention_over_all_pages_is_attention():
    rng = np.random.default_rng(3)
    kc, vc = _cache(rng)
    table, lens, q = rng.permutation(30)[:12].reshape(2, 6), [23, 9], rng.standard_normal((2, 4, 8))
    sel = np.tile(np.arange(6), (2, 2, 1))
    o, lse = longctx.select_attn_decode(q, kc, vc, table, lens, sel, 0.3)
    wo, wl = paged.paged_attn_decode(q, kc, vc, table, lens, 0.3)
    np.testing.assert_allclose(o, wo, rtol=1e-12)
    np.testing.assert_allclose(lse, wl, rtol=1e-12)
    # page 1 and the partly filled last one
    o, lse = longctx.select_attn_decode(q[:1], kc, vc, table[:1], lens[:1], [[[1, 5], [5, -1]]], 0.3)
    wo, wl = paged.paged_attn_decode(q[:1], kc, vc, table[:1, [1, 5]], [7], 0.3)
    np.testing.assert_allclose(o[0, :2], wo[0, :2], rtol=1e-12)
    wo, wl = paged.paged_attn_decode(q[:1], kc, vc, table[:1, [5]], [3], 0.3)
    np.testing.assert_allclose(o[0, 2:], wo[0, 2:], rtol=1e-12)
    np.testing.assert_allclose(lse[0, 2:], wl[0, 2:], rtol=1e-12)


def test_weights_add_up_to_one_a_row_and_head():
    rng = np.random.default_rng(4)
    kc, vc = _cache(rng)
    table = rng.permutation(30)[:12].reshape(2, 6)
    old, lens = np.array([7, 0]), np.array([11, 9])
    starts = [0, 4, 13]
    pos = np.concatenate([np.arange(7, 11), np.arange(0, 9)])
    q = rng.standard_normal((13, 4, 8))
    req = np.repeat([0, 1], [4, 9])
    _, lse = paged.paged_attn_decode(q, kc, vc, table[req], pos + 1, 0.3)
    m = longctx.mass_update(q, kc, lse, np.full((30, 2, 4), 0.5), table, starts, pos, old, lens, 0.3)
    for r in range(2):
        j = np.arange(lens[r])
        got = m[table[r, j // 4], :, j % 4].sum(0) - 0.5 * old[r]
        np.testing.assert_allclose(got, (lens[r] - old[r]) * 2, rtol=1e-12)      # rows times heads of a kv head
    # the first token of a prompt gathers the whole weight of its own row; rows out of place add nothing
    one = longctx.mass_update(q[4:5], kc, lse[4:5], np.zeros((30, 2, 4)), table[1:], [0, 1], [0], [0], [9], 0.3)
    assert one[table[1, 0], 0, 0] > 0.999 * 2 and one.sum() < 4.001
    none = longctx.mass_update(q[4:5], kc, lse[4:5], np.ones((30, 2, 4)), table[1:], [0, 1], [9], [9], [9], 0.3)
    assert (none == 1).all()


def test_evict_hand_case():
    k = np.arange(24.0).reshape(3, 4, 2, 1)
    mass = np.zeros((3, 2, 4))
    table = np.array([[2, 0, 1]])
    m = {0: [5, 1, 7, 1, 9, 0, 3, 2, 0, 0], 1: [0] * 10}
    for g in (0, 1):
        for j in range(10):
            mass[table[0, j // 4], g, j % 4] = m[g][j]
    k2, v2, m2, n, kept = longctx.evict(k, -k, mass, table, [10], 5, 2)
    assert n.tolist() == [5] and kept.tolist() == [[[0, 2, 4, 8, 9], [0, 1, 2, 8, 9]]]
    at = lambda j: (table[0, j // 4], j % 4)  # noqa: E731
    for g in (0, 1):
        for i, j in enumerate(kept[0, g]):
            assert k2[at(i)][g] == k[at(j)][g] and v2[at(i)][g] == -k[at(j)][g]
            assert m2[at(i)[0], g, at(i)[1]] == m[g][j]
        for j in range(5, 12):
            assert k2[at(j)][g] == k[at(j)][g]
    *_, n, kept = longctx.evict(k, -k, mass, table, [4], 5, 2)
    assert n.tolist() == [4] and kept[0, 0].tolist() == [0, 1, 2, 3, -1]
