"""fp64 CPU oracle for the paged-attention operators -- TEST INFRASTRUCTURE.

Plain numpy, from the operators' definitions, request by request and head by head; it
imports nothing from the product package and shares no code with it.  What pins it is in
tests/test_oracle_paged_pins.py.
"""
from __future__ import annotations

import numpy as np


def pages_step(len_old, len_new, table, free_ring, ring, page_size, n_tokens):
    """One scheduling step with Python lists: the free pages as a queue.  Returns a dict with
    block_table, free_ring, ring, len, starts, request, positions, slots, denied."""
    table = np.array(table, np.int64)
    batch, max_pages = table.shape
    n = len(free_ring)
    head, free = int(ring[0]), int(ring[1])
    queue = [int(free_ring[(head + i) % n]) for i in range(free)]
    place = np.array(free_ring, np.int64)
    tail = head + free                       # where the next page given back goes
    given, length, request, positions, slots, starts = [], [], [], [], [], [0]
    needed = used = denied = 0
    for r in range(batch):
        lo, hi = max(int(len_old[r]), 0), max(int(len_new[r]), 0)
        have, want = -(-lo // page_size), -(-hi // page_size)
        refuse = want > max_pages
        if not refuse and want > have:
            needed += want - have
            refuse = needed > free
        if refuse:
            denied += 1
        elif want > have:
            for c in range(have, want):
                table[r, c] = queue[used]
                used += 1
        else:
            given += [int(p) for p in table[r, want:have]]
        length.append(lo if refuse else hi)
        for p in range(lo, hi):
            request.append(r)
            positions.append(p)
            slots.append(-1 if refuse else int(table[r, p // page_size]) * page_size + p % page_size)
        starts.append(len(request))
    for p in given:
        place[tail % n] = p
        tail += 1
    pad = max(0, n_tokens - len(request))
    cut = lambda v: np.array((v + [-1] * pad)[:n_tokens], np.int64)  # noqa: E731
    return dict(block_table=table, free_ring=place, ring=np.array([(head + used) % n, free - used + len(given)]),
                len=np.array(length), starts=np.array(starts), request=cut(request), positions=cut(positions),
                slots=cut(slots), denied=np.array([denied]))


def _angles(positions, inv_freq):
    return np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]


def _pairs(rot, interleaved):
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def qk_norm_rope(x, w, inv_freq, positions, eps=1e-6, interleaved=False):
    """Heads x (T, H, d) normed with w (d,) (None: not normed) and rotated."""
    x = np.asarray(x, np.float64)
    y = x.copy() if w is None else x * np.asarray(w, np.float64) / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    th = _angles(positions, inv_freq)[:, None]
    a, b = _pairs(2 * th.shape[-1], interleaved)
    out = y.copy()
    out[..., a] = y[..., a] * np.cos(th) - y[..., b] * np.sin(th)
    out[..., b] = y[..., b] * np.cos(th) + y[..., a] * np.sin(th)
    return out


def qk_norm_rope_bwd(x, w, inv_freq, positions, dout, eps=1e-6, interleaved=False):
    """(dx, dw) of qk_norm_rope for the cotangent dout; dw is None without a norm."""
    x, g = np.asarray(x, np.float64), np.array(dout, np.float64)
    th = _angles(positions, inv_freq)[:, None]
    a, b = _pairs(2 * th.shape[-1], interleaved)
    ga, gb = g[..., a].copy(), g[..., b].copy()
    g[..., a] = ga * np.cos(th) + gb * np.sin(th)
    g[..., b] = gb * np.cos(th) - ga * np.sin(th)
    if w is None:
        return g, None
    w = np.asarray(w, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dx = r * (w * g - n * (w * g * n).mean(-1, keepdims=True))
    return dx, (g * n).sum((0, 1))


def paged_attn_decode(q, k_cache, v_cache, table, lens, scale, window=0):
    """q (B, H, d); caches (pages, page_size, Hk, d) holding the values themselves; table
    (B, cols); lens (B,).  Returns o (B, H, d) and lse (B, H)."""
    q, table = np.asarray(q, np.float64), np.asarray(table)
    B, H, d = q.shape
    n_pages, ps, Hk, _ = k_cache.shape
    o, lse = np.zeros((B, H, d)), np.full((B, H), -np.inf)
    for r in range(B):
        n = min(max(int(lens[r]), 0), table.shape[1] * ps)
        toks = [(int(table[r, j // ps]), j % ps) for j in range(max(0, n - window) if window > 0 else 0, n)]
        toks = [t for t in toks if 0 <= t[0] < n_pages]
        if not toks:
            continue
        p, i = np.array(toks).T
        for h in range(H):
            g = h * Hk // H
            s = scale * (np.asarray(k_cache[p, i, g], np.float64) @ q[r, h])
            top = s.max()
            if top == -np.inf:
                continue
            e = np.exp(s - top)
            o[r, h] = e @ np.asarray(v_cache[p, i, g], np.float64) / e.sum()
            lse[r, h] = top + np.log(e.sum())
    return o, lse
