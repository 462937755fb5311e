"""fp64 CPU oracle for the long-context operators of a paged cache -- TEST INFRASTRUCTURE.

Plain numpy, from the operators' definitions, request by request and head by head; it
imports nothing from the product package and shares no code with it.  What pins it is in
tests/test_oracle_longctx_pins.py.
"""
from __future__ import annotations

import numpy as np


def _tokens(table, n, ps, n_pages):
    """(token, page, place) of the tokens below n that stand on a page of the cache."""
    n = min(max(int(n), 0), len(table) * ps)
    got = [(j, int(table[j // ps]), j % ps) for j in range(n)]
    return [t for t in got if 0 <= t[1] < n_pages]


def _attend(q, k, v, scale):
    """One query over rows k, v: (o, lse)."""
    if len(k) == 0:
        return np.zeros_like(q), -np.inf
    s = scale * (k @ q)
    top = s.max()
    if top == -np.inf:
        return np.zeros_like(q), -np.inf
    e = np.exp(s - top)
    return e @ v / e.sum(), top + np.log(e.sum())


def prefix_attn_decode(q, k_cache, v_cache, prefix, prefix_table, prefix_lens, table, lens, scale):
    """q (B, H, d); caches (pages, page_size, Hk, d) holding the values themselves."""
    q = np.asarray(q, np.float64)
    B, H, _ = q.shape
    n_pages, ps, Hk, _ = k_cache.shape
    o, lse = np.zeros(q.shape), np.full((B, H), -np.inf)
    for r in range(B):
        toks = []
        if 0 <= prefix[r] < len(prefix_lens):
            toks += _tokens(prefix_table[prefix[r]], prefix_lens[prefix[r]], ps, n_pages)
        toks += _tokens(table[r], lens[r], ps, n_pages)
        p, i = [t[1] for t in toks], [t[2] for t in toks]
        for h in range(H):
            g = h * Hk // H
            o[r, h], lse[r, h] = _attend(q[r, h], np.asarray(k_cache[p, i, g], np.float64).reshape(-1, q.shape[2]),
                                         np.asarray(v_cache[p, i, g], np.float64).reshape(-1, q.shape[2]), scale)
    return o, lse


def page_bounds(k_cache, bounds, table, len_old, lens):
    """bounds (pages, Hk, 2, d) after the tokens [len_old, lens) have entered k_cache."""
    b = np.array(bounds, np.float64)
    n_pages, ps = k_cache.shape[:2]
    for r in range(len(lens)):
        start = min(max(int(len_old[r]), 0), len(table[r]) * ps)
        for j, p, i in _tokens(table[r], lens[r], ps, n_pages):
            if j < start:
                continue
            k = np.asarray(k_cache[p, i], np.float64)
            if i == 0:
                b[p, :, 0], b[p, :, 1] = k, k
            else:
                b[p, :, 0], b[p, :, 1] = np.minimum(b[p, :, 0], k), np.maximum(b[p, :, 1], k)
    return b


def page_scores(q, bounds, table, n, h_of_g):
    """Scores of the first n pages of one row for the query heads h_of_g (g -> heads), (Hk, n) fp32."""
    out = np.full((len(h_of_g), n), -np.inf, np.float32)
    for g, heads in enumerate(h_of_g):
        for i in range(n):
            if not 0 <= table[i] < len(bounds):
                continue
            lo, hi = np.asarray(bounds[table[i], g], np.float64)
            s = [np.float32((np.maximum(q[h], 0) * hi + np.minimum(q[h], 0) * lo).sum()) for h in heads]
            out[g, i] = np.max(s)                # (NaN if one is)
    return out


def page_select(q, bounds, table, lens, page_size, top_k, first, last):
    q = np.asarray(q, np.float64)
    B, H, _ = q.shape
    Hk = bounds.shape[1]
    out = np.full((B, Hk, top_k), -1, np.int64)
    for r in range(B):
        n = -(-min(max(int(lens[r]), 0), table.shape[1] * page_size) // page_size)
        heads = [range(g * (H // Hk), (g + 1) * (H // Hk)) for g in range(Hk)]
        sc = page_scores(q[r], bounds, table[r], n, heads) if n > top_k else None
        for g in range(Hk):
            if n <= top_k:
                out[r, g, :n] = np.arange(n)
                continue
            mid = range(first, n - last)
            order = sorted(mid, key=lambda i: (not np.isnan(sc[g, i]), 0 if np.isnan(sc[g, i]) else -sc[g, i], i))
            out[r, g] = sorted(list(range(first)) + list(range(n - last, n)) + order[:top_k - first - last])
    return out


def select_attn_decode(q, k_cache, v_cache, table, lens, selected, scale):
    q = np.asarray(q, np.float64)
    B, H, d = q.shape
    n_pages, ps, Hk, _ = k_cache.shape
    o, lse = np.zeros(q.shape), np.full((B, H), -np.inf)
    for r in range(B):
        at = {}
        for j, p, i in _tokens(table[r], lens[r], ps, n_pages):
            at.setdefault(j // ps, []).append((p, i))
        held = -(-min(max(int(lens[r]), 0), table.shape[1] * ps) // ps)
        for h in range(H):
            g = h * Hk // H
            toks = [t for s in selected[r][g][:held] for t in at.get(int(s), [])]
            p, i = [t[0] for t in toks], [t[1] for t in toks]
            o[r, h], lse[r, h] = _attend(q[r, h], np.asarray(k_cache[p, i, g], np.float64).reshape(-1, d),
                                         np.asarray(v_cache[p, i, g], np.float64).reshape(-1, d), scale)
    return o, lse


def mass_update(q, k_cache, lse, mass, table, starts, positions, len_old, lens, scale):
    """mass (pages, Hk, page_size) after a step."""
    q, m = np.asarray(q, np.float64), np.array(mass, np.float64)
    T, H, _ = q.shape
    n_pages, ps, Hk, _ = k_cache.shape
    for r in range(len(lens)):
        toks = _tokens(table[r], lens[r], ps, n_pages)
        n = min(max(int(lens[r]), 0), table.shape[1] * ps)
        s0 = min(max(int(starts[r]), 0), T)
        rows = [t for t in range(s0, min(max(int(starts[r + 1]), s0), T)) if 0 <= positions[t] < n]
        for j, p, i in toks:
            for g in range(Hk):
                w = 0.0
                for t in rows:
                    if j > positions[t]:
                        continue
                    for h in range(g * (H // Hk), (g + 1) * (H // Hk)):
                        if lse[t, h] != -np.inf:
                            w += np.exp(scale * (q[t, h] @ np.asarray(k_cache[p, i, g], np.float64)) - float(lse[t, h]))
                m[p, g, i] = w + (m[p, g, i] if j < len_old[r] else 0.0)
    return m


def evict(k_cache, v_cache, mass, table, lens, budget, recent):
    """(k_cache, v_cache, mass, len, kept) after the eviction; the caches may hold any values."""
    k, v, m = k_cache.copy(), v_cache.copy(), np.array(mass)
    n_pages, ps, Hk = k.shape[:3]
    B = len(lens)
    length, kept = np.zeros(B, np.int64), np.full((B, Hk, budget), -1, np.int64)
    for r in range(B):
        n = min(max(int(lens[r]), 0), table.shape[1] * ps)
        length[r] = min(n, budget)
        if n <= budget:
            kept[r, :, :n] = np.arange(n)
            continue
        page = lambda j: int(table[r][j // ps]) if 0 <= table[r][j // ps] < n_pages else -1  # noqa: E731
        for g in range(Hk):
            def rank(j):
                x = float(mass[page(j), g, j % ps]) if page(j) >= 0 else -np.inf
                return (0, 0.0, j) if np.isnan(x) else (1, -x, j)
            best = sorted(range(n - recent), key=rank)[:budget - recent]
            kept[r, g] = sorted(best) + list(range(n - recent, n))
            for i, j in enumerate(kept[r, g]):
                if page(i) >= 0 and page(j) >= 0:
                    k[page(i), i % ps, g] = k_cache[page(j), j % ps, g]
                    v[page(i), i % ps, g] = v_cache[page(j), j % ps, g]
                    m[page(i), g, i % ps] = mass[page(j), g, j % ps]
    return k, v, m, length, kept
