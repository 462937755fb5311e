"""Measured cases of the operators that keep long contexts cheap to serve from a paged cache.

Six operators: attention of one new token a row where rows share a long prefix (``prefix``);
the smallest and largest keys of each page (``bounds``), the choice of each row's pages by
them (``select``) and attention over the chosen pages alone (``sparse``); the attention weight
that each cached token gathers (``mass``), and keeping the tokens that gathered most
(``evict``).

``own`` picks what ``run`` does: the plain torch form, or the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f8": 1}
CACHE_SCALE = 0.03125     # an 8-bit cache holds k / CACHE_SCALE, v / CACHE_SCALE


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # a batch of answers under one long common prompt
        {"name": "prefix 64 long", "op": "prefix", "batch": 64, "prefixes": 1, "plen": 16384, "len": 512, "heads": 32,
         "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 16, "layout": "nhd"},
        # a few requests of three programs, each with a prompt of its own, 8-bit cache
        {"name": "prefix few f8", "op": "prefix", "batch": 13, "prefixes": 3, "plen": 4001, "len": 100, "heads": 20,
         "kv_heads": 4, "dim": 128, "cache": "f8", "page": 64, "layout": "hnd"},
        # a decode step of a full batch: each request's last page has one more key
        {"name": "bounds decode 256", "op": "bounds", "batch": 256, "old": 4096, "grow": 1, "kv_heads": 8, "dim": 128,
         "cache": "bf16", "page": 16, "layout": "nhd"},
        # prompts that enter an 8-bit cache
        {"name": "bounds prompts f8", "op": "bounds", "batch": 8, "old": 0, "grow": 8192, "kv_heads": 8, "dim": 128,
         "cache": "f8", "page": 64, "layout": "hnd"},
        # long answers: 128 pages of up to 2048 for each row and kv head
        {"name": "select long", "op": "select", "batch": 32, "len": 32768, "heads": 32, "kv_heads": 8, "dim": 128,
         "cache": "bf16", "page": 16, "layout": "nhd", "top": 128, "first": 1, "last": 4},
        # a few rows of odd sizes, fp32
        {"name": "select odd f32", "op": "select", "batch": 5, "len": 3001, "heads": 6, "kv_heads": 3, "dim": 72,
         "cache": "f32", "page": 24, "layout": "nhd", "top": 17, "first": 0, "last": 1},
        # attention over the pages of the long case: 2048 tokens a row
        {"name": "sparse long", "op": "sparse", "batch": 32, "len": 32768, "heads": 32, "kv_heads": 8, "dim": 128,
         "cache": "bf16", "page": 16, "layout": "nhd", "top": 128, "first": 1, "last": 4},
        # one request alone, 8-bit cache with wide pages: latency
        {"name": "sparse one f8", "op": "sparse", "batch": 1, "len": 20011, "heads": 16, "kv_heads": 2, "dim": 128,
         "cache": "f8", "page": 64, "layout": "hnd", "top": 32, "first": 1, "last": 2},
        # a decode step of a batch in the middle of its answers
        {"name": "mass decode 64", "op": "mass", "batch": 64, "old": 8192, "grow": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "cache": "bf16", "page": 16, "layout": "nhd"},
        # prompts of different lengths: every query's weights
        {"name": "mass prompts", "op": "mass", "batch": 4, "old": 0, "grow": 2048, "heads": 32, "kv_heads": 8, "dim": 128,
         "cache": "bf16", "page": 16, "layout": "nhd"},
        # a batch whose answers have outgrown their budget by a few pages
        {"name": "evict decode 64", "op": "evict", "batch": 64, "len": 4160, "ragged": False, "budget": 4096, "recent": 512,
         "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 16, "layout": "nhd"},
        # long prompts cut to a budget, 8-bit cache, odd lengths
        {"name": "evict prompts f8", "op": "evict", "batch": 3, "len": 16001, "ragged": True, "budget": 2048, "recent": 63,
         "kv_heads": 4, "dim": 128, "cache": "f8", "page": 64, "layout": "hnd"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "bounds", "select", "sparse", "mass", "evict"])
    kv = rng.choice([1, 2, 3, 4, 8])
    case = {"op": op, "kv_heads": kv, "cache": rng.choice(["bf16", "bf16", "f8", "f32"]),
            "dim": rng.choice([64, 80, 96, 128, 128, 192, 256]), "layout": rng.choice(["nhd", "hnd"])}
    d = case["dim"]
    if op not in ("bounds", "evict"):
        case["heads"] = kv * rng.choice([1, 2, 3, 4, 5, 8])
    if op == "prefix":
        case.update(batch=_log(rng, 2, 128), page=rng.choice([8, 16, 16, 24, 64, 128]), len=_log(rng, 1, 2048))
        case["prefixes"] = rng.choice([1, 1, 2, 3, 5])
        # score products of the whole batch, and the cache's elements
        room = min(8e9 * (0.25 if case["cache"] == "f32" else 1.0) / (case["batch"] * case["heads"] * d),
                   4e8 / (case["prefixes"] * kv * d))
        case["plen"] = max(1, min(_log(rng, 16, 65536), int(room)))
        case["len"] = max(1, min(case["len"], int(2e8 / (case["batch"] * kv * d))))
        return case
    if op == "bounds":
        grow = rng.choice([1, 1, _log(rng, 2, 8192)])
        case.update(batch=_log(rng, 1, 256), old=rng.choice([0, _log(rng, 1, 8192)]), grow=grow,
                    page=rng.choice([1, 8, 16, 24, 64, 128]))
        case["batch"] = max(1, min(case["batch"], int(1.2e8 / ((case["old"] + grow) * kv * d))))
        return case
    if op in ("select", "sparse"):
        case.update(batch=_log(rng, 1, 64), page=rng.choice([8, 16, 16, 24, 64, 128]), len=_log(rng, 64, 131072),
                    first=rng.choice([0, 1, 2]), last=rng.choice([0, 1, 4]))
        case["top"] = case["first"] + case["last"] + _log(rng, 1, 256)
        case["batch"] = max(1, min(case["batch"], int(2.4e8 / (case["len"] * kv * d))))
        if op == "sparse":
            case["top"] = min(case["top"], max(7, 4096 // case["page"]))
        return case
    if op == "mass":
        case.update(batch=_log(rng, 1, 128), page=rng.choice([1, 8, 16, 16, 24, 64]))
        if rng.random() < 0.6:
            case.update(old=_log(rng, 1, 32768), grow=1)
            case["batch"] = max(1, min(case["batch"], int(5e8 / ((case["old"] + 1) * kv * d))))
        else:
            case.update(old=rng.choice([0, _log(rng, 1, 2048)]), grow=_log(rng, 2, 2048))
            pairs = case["grow"] * (case["old"] + case["grow"]) * case["heads"]
            case["batch"] = max(1, min(case["batch"], 8, int(4e8 / pairs)))
        return case
    case.update(batch=_log(rng, 1, 64), page=rng.choice([8, 16, 24, 64]), len=_log(rng, 2, 16384), ragged=rng.random() < 0.7)
    case["budget"] = max(1, int(case["len"] * rng.choice([0.125, 0.5, 0.9, 0.98])))
    case["recent"] = int(case["budget"] * rng.choice([0.0, 0.1, 0.5, 1.0]))
    case["batch"] = max(1, min(case["batch"], int(2e8 / (case["len"] * kv * d))))
    return case


def _spread(n, top):
    """n lengths spread over 1..top, with one idle place among more than three."""
    part = np.modf(0.5 + 0.6180339887498949 * np.arange(n))[0]
    got = 1 + (part * (top - 1)).astype(np.int64)
    if n >= 4:
        got[3] = 0
    return got


def _lengths(case):
    """Tokens that each request holds, and (where some are new) held before."""
    n, op = case["batch"], case["op"]
    if op in ("bounds", "mass"):
        part = np.modf(0.5 + 0.6180339887498949 * np.arange(n))[0]
        old = (case["old"] * (0.5 + 0.5 * part)).astype(np.int64)
        new = np.ones_like(old) if case["grow"] == 1 else 1 + (part * (case["grow"] - 1)).astype(np.int64)
        if n >= 4:
            new[3] = 0
        return old + new, old
    if op == "evict" and not case["ragged"]:
        return np.full(n, case["len"], dtype=np.int64), None
    return _spread(n, case["len"]), None


def _prefixes(case):
    """The prefixes' lengths, and for each row its prefix (-1: none), rows of one next to each other."""
    n = case["prefixes"]
    lens = np.maximum(1, case["plen"] - np.arange(n) * (case["plen"] // (2 * n)))
    of = np.arange(case["batch"]) * n // case["batch"]
    if n > 1:
        of[-1] = -1
    return lens, of


# ----------------------------------------------------------------- inputs ----
def _cache(case, pages, g):
    """A (pages, page, kv_heads, dim) view of a cache in the case's layout."""
    dtype, hk, d, ps = DTYPES[case["cache"]], case["kv_heads"], case["dim"], case["page"]
    shape = (pages, ps, hk, d) if case["layout"] == "nhd" else (pages, hk, ps, d)
    c = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if case["cache"] == "f32" else torch.bfloat16)
    c = c.div_(CACHE_SCALE).to(dtype) if case["cache"] == "f8" else c
    return c if case["layout"] == "nhd" else c.permute(0, 2, 1, 3)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 32))
    s, op, ps, hk, d = dict(case), case["op"], case["page"], case["kv_heads"], case["dim"]
    s["cache_scale"] = CACHE_SCALE if case["cache"] == "f8" else 1.0
    s["scale"] = d ** -0.5
    heads_type = torch.float32 if case["cache"] == "f32" else torch.bfloat16

    def ints(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", torch.int32)

    def randn(*shape, dtype=heads_type):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    # each request's pages anywhere in the cache
    lens, old = _lengths(case)
    held = lens if op != "prefix" else np.concatenate([lens, _prefixes(case)[0]])
    have = -(-held // ps)
    total = int(have.sum()) + 3
    table = np.full((len(held), max(1, int(have.max()))), -1, dtype=np.int64)
    table[np.arange(table.shape[1])[None] < have[:, None]] = rs.permutation(total)[:int(have.sum())]
    s["lens"] = ints(lens)
    if op == "prefix":
        plens, of = _prefixes(case)
        cols = max(1, int(have[:len(lens)].max()))
        s["prefix_table"], table = ints(table[len(lens):]), table[:len(lens), :cols]
        s["prefix_lens"], s["prefix"] = ints(plens), ints(of)
    s["table"] = ints(table)
    if op in ("bounds", "mass"):
        s["len_old"] = ints(old)
    if op != "select":
        s["k_cache"] = _cache(case, total, g)
    if op in ("prefix", "sparse", "evict"):
        s["v_cache"] = _cache(case, total, g)
    if op in ("prefix", "select", "sparse"):
        s["q"] = randn(case["batch"], case["heads"], d)
    if op == "bounds":
        # what a page that holds tokens already has; pages that new tokens open hold anything
        s["bounds"] = torch.empty((total, hk, 2, d), device="cuda", dtype=DTYPES[case["cache"]])
        b = randn(total, hk, 2, d, dtype=torch.float32).sort(2).values / s["cache_scale"]
        s["bounds"].copy_(b)
    if op == "select":
        # of keys with a common part and a part of each page: some pages matter more, as they do in text
        b = (randn(total, hk, 2, d, dtype=torch.float32).sort(2).values + 0.5 * randn(total, hk, 1, d, dtype=torch.float32))
        s["bounds"] = (b / s["cache_scale"]).to(DTYPES[case["cache"]])
    if op == "sparse":
        n = torch.from_numpy(have).cuda()
        s["selected"] = _pick(randn(case["batch"], hk, table.shape[1], dtype=torch.float32), n, case)
    if op == "mass":
        rows = lens - old
        starts = np.concatenate([[0], np.cumsum(rows)])
        s["n_tokens"], s["most_rows"] = int(starts[-1]), int(rows.max())
        s["starts"] = ints(starts)
        s["positions"] = ints(np.concatenate([np.arange(a, b) for a, b in zip(old, lens)]))
        s["q"] = randn(s["n_tokens"], case["heads"], d)
        s["mass"] = torch.rand((total, hk, ps), generator=g, device="cuda")
        s["lse"] = _plain_lse(s)
    if op == "evict":
        # a few tokens gather most of the weight, many next to none
        s["mass"] = torch.exp(2.5 * randn(total, hk, ps, dtype=torch.float32))
    return s


# ------------------------------------------------------------ plain forms ----
def _values(cache, page, at, s):
    """Rows of a cache, in fp32."""
    if cache.dtype == torch.float8_e4m3fn:
        return cache.view(torch.uint8)[page, at].view(cache.dtype).float() * s["cache_scale"]
    return cache[page, at].float()


def _places(table, lens, n, ps):
    """(page, place, held) of the tokens 0..n-1 of each row."""
    tok = torch.arange(n, device=table.device)
    held = tok < lens.long()[:, None]
    page = torch.where(held, table[:, tok // ps].long(), 0)
    return page, (tok % ps).expand(len(table), -1), held


def _softmax_sum(sc, v):
    """(unnormalised output, maximum, sum) of scores (..., tokens) with values (..., tokens, dim)."""
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(sc - top)
    return torch.matmul(p, v), top, p.sum(-1, keepdim=True)


def _plain_prefix(s):
    q, hk = s["q"], s["kv_heads"]
    b, h, d = q.shape
    qg = q.float().view(b, hk, h // hk, d)
    page, at, held = _places(s["table"], s["lens"], s["table"].shape[1] * s["page"], s["page"])
    k = _values(s["k_cache"], page, at, s)
    sc = (torch.matmul(qg, k.permute(0, 2, 3, 1)) * s["scale"]).masked_fill(~held[:, None, None], -math.inf)
    v = _values(s["v_cache"], page, at, s).masked_fill(~held[..., None, None], 0.0)
    o, top, mass = _softmax_sum(sc, v.transpose(1, 2))
    # each prefix's tokens once, for all of its rows
    lens, of = _prefixes(s)
    for p, n in enumerate(lens.tolist()):
        rows = np.nonzero(of == p)[0]
        if not len(rows):
            continue
        r0, r1 = int(rows[0]), int(rows[-1]) + 1
        tok = torch.arange(n, device=q.device)
        page, at = s["prefix_table"][p, tok // s["page"]].long(), tok % s["page"]
        k = _values(s["k_cache"], page, at, s).permute(1, 2, 0)
        sc = torch.matmul(qg[r0:r1].transpose(0, 1).reshape(hk, -1, d), k) * s["scale"]
        v = _values(s["v_cache"], page, at, s).transpose(0, 1)
        o2, top2, mass2 = (x.view(hk, r1 - r0, h // hk, -1).transpose(0, 1) for x in _softmax_sum(sc, v))
        both = torch.maximum(top[r0:r1], top2)
        f1, f2 = torch.exp(top[r0:r1] - both) * (mass[r0:r1] > 0), torch.exp(top2 - both)
        both = torch.where(mass[r0:r1] > 0, both, top2)
        f2 = torch.where(mass[r0:r1] > 0, f2, 1.0)
        o[r0:r1] = o[r0:r1] * f1 + o2 * f2
        mass[r0:r1] = mass[r0:r1] * f1 + mass2 * f2
        top[r0:r1] = both
    out = o / torch.where(mass > 0, mass, 1.0)
    return {"o": out.view(b, h, d).to(q.dtype), "lse": (top + torch.log(mass)).view(b, h)}


def _plain_bounds(s):
    ps = s["page"]
    lens, old = _lengths(s)
    first, last = old // ps, -(-lens // ps)
    n = np.where(lens > old, last - first, 0)
    r = torch.from_numpy(np.repeat(np.arange(len(lens)), n)).cuda()
    i = torch.from_numpy(np.concatenate([np.arange(a, a + c) for a, c in zip(first, n)])).cuda()
    lo, hi = s["len_old"].long()[r][:, None], s["lens"].long()[r][:, None]
    tok = i[:, None] * ps + torch.arange(ps, device=r.device)
    new = ((tok >= lo) & (tok < hi))[..., None, None]
    page = s["table"][r, i].long()
    cache = s["k_cache"]
    k = (cache.view(torch.uint8)[page].view(cache.dtype) if s["cache"] == "f8" else cache[page]).float()
    low, high = k.masked_fill(~new, math.inf).amin(1), k.masked_fill(~new, -math.inf).amax(1)
    b = s["bounds"]
    had = ((b.view(torch.uint8)[page].view(b.dtype) if s["cache"] == "f8" else b[page])).float()
    more = (i[:, None] * ps < lo)[..., None]
    low = torch.where(more, torch.minimum(low, had[:, :, 0]), low)
    high = torch.where(more, torch.maximum(high, had[:, :, 1]), high)
    new_b = torch.stack([low, high], 2).to(b.dtype)
    if s["cache"] == "f8":
        b.view(torch.uint8)[page] = new_b.view(torch.uint8)
    else:
        b[page] = new_b
    return {"bounds": b}


def _pick(score, n, case):
    """The pages of each (row, kv head): the first, the last and the best scored ones, `top` in all,
    in order; -1 behind the last.  n (rows,): pages that a row has."""
    i = torch.arange(score.shape[-1], device=score.device)
    n = n[:, None, None]
    forced = (i < case["first"]) | (i >= n - case["last"])
    key = torch.where(forced, math.inf, score).masked_fill(i >= n, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    keep = torch.zeros_like(forced.expand_as(score))
    keep.scatter_(-1, order[..., :case["top"]], True)
    keep = keep & (i < n)
    got = torch.where(keep, i, score.shape[-1]).sort(-1).values
    got = torch.nn.functional.pad(got, (0, max(0, case["top"] - got.shape[-1])), value=score.shape[-1])[..., :case["top"]]
    return torch.where(got < score.shape[-1], got, -1).int()


def _plain_select(s):
    # (in 64 bits: the order of scores that lie close together decides)
    b, h, d = s["q"].shape
    hk, cols = s["kv_heads"], s["table"].shape[1]
    score = torch.full((b, hk, cols), -math.inf, device="cuda")
    n = (s["lens"].long() + s["page"] - 1) // s["page"]
    bounds = s["bounds"]
    for r in range(b):
        page = s["table"][r].long().clamp(min=0)
        x = (bounds.view(torch.uint8)[page].view(bounds.dtype) if s["cache"] == "f8" else bounds[page]).double()
        x = x.permute(2, 1, 3, 0)                   # (2, kv head, dim, page)
        q = s["q"][r].double().view(hk, h // hk, d)
        both = torch.matmul(q.clamp(max=0.0), x[0]) + torch.matmul(q.clamp(min=0.0), x[1])
        score[r] = both.float().amax(1)
    return {"selected": _pick(score, n, s)}


def _plain_sparse(s):
    q, hk, ps, top = s["q"], s["kv_heads"], s["page"], s["top"]
    b, h, d = q.shape
    listed_page = s["selected"].long()                                     # (row, kv head, entry)
    tok = listed_page[..., None] * ps + torch.arange(ps, device=q.device)
    held = ((listed_page >= 0)[..., None] & (tok < s["lens"].long()[:, None, None, None])).view(b, hk, top * ps)
    page = torch.gather(s["table"].long(), 1, listed_page.clamp(min=0).view(b, -1)).view(b, hk, top, 1)
    page = page.expand(-1, -1, -1, ps).reshape(b, hk, top * ps).clamp(min=0)
    at = torch.arange(ps, device=q.device).repeat(top).expand(b, hk, -1)
    head = torch.arange(hk, device=q.device)[None, :, None]

    def rows(cache):
        if s["cache"] == "f8":
            return cache.view(torch.uint8)[page, at, head].view(cache.dtype).float() * s["cache_scale"]
        return cache[page, at, head].float()

    sc = torch.matmul(q.float().view(b, hk, h // hk, d), rows(s["k_cache"]).transpose(-1, -2)) * s["scale"]
    sc = sc.masked_fill(~held[:, :, None], -math.inf)
    o, most, mass = _softmax_sum(sc, rows(s["v_cache"]).masked_fill(~held[..., None], 0.0))
    o = o / torch.where(mass > 0, mass, 1.0)
    return {"o": o.view(b, h, d).to(q.dtype), "lse": (most + torch.log(mass)).view(b, h)}


def _row_scores(s, rows):
    """Scores of each request's rows [rows) over its tokens: (request, kv head, rows * group, tokens), -inf where
    a row does not see a token, and the rows' places among all rows (clamped) with the rows that are there."""
    b, hk, ps = s["batch"], s["kv_heads"], s["page"]
    h, d = s["q"].shape[1:]
    page, at, held = _places(s["table"], s["lens"], s["table"].shape[1] * ps, ps)
    k = _values(s["k_cache"], page, at, s).permute(0, 2, 3, 1)
    first, end = s["starts"][:-1].long()[:, None], s["starts"][1:].long()[:, None]
    t = first + torch.arange(rows[0], rows[1], device=k.device)
    there = t < end
    t = t.clamp(max=s["n_tokens"] - 1)
    pos = torch.where(there, s["positions"].long()[t], -1)
    q = s["q"][t].float().view(b, t.shape[1], hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    sc = (torch.matmul(q, k) * s["scale"]).view(b, hk, t.shape[1], h // hk, -1)
    sees = torch.arange(sc.shape[-1], device=k.device) <= pos[..., None]
    return sc.masked_fill_(~sees[:, None, :, None], -math.inf), t, there, (page, at, held)


def _chunks(s):
    """Rows at a time, so that their scores take 2 GB at most."""
    per = s["batch"] * s["heads"] * s["table"].shape[1] * s["page"] * 4
    step = max(1, int(2e9 // per))
    return [(i, min(i + step, s["most_rows"])) for i in range(0, s["most_rows"], step)]


def _plain_lse(s):
    lse = torch.zeros((s["n_tokens"], s["heads"]), device="cuda")
    for rows in _chunks(s):
        sc, t, there, _ = _row_scores(s, rows)
        got = torch.logsumexp(sc, -1).transpose(1, 2).reshape(*t.shape, -1)
        lse[t[there]] = got[there]
    return lse


def _plain_mass(s):
    total = None
    for rows in _chunks(s):
        sc, t, there, (page, at, held) = _row_scores(s, rows)
        b, hk, n, group, tokens = sc.shape
        lse = s["lse"][t].view(b, n, hk, group).transpose(1, 2)[..., None]
        w = torch.exp(sc - lse).sum((2, 3))
        total = w if total is None else total + w
    r, j = held.nonzero(as_tuple=True)
    p, i = page[r, j], at[r, j]
    was = torch.where((j < s["len_old"].long()[r])[:, None], s["mass"][p, :, i], 0.0)
    s["mass"][p, :, i] = was + total[r, :, j]
    return {"mass": s["mass"]}


def _plain_evict(s):
    ps, hk, budget, recent = s["page"], s["kv_heads"], s["budget"], s["recent"]
    lens = s["lens"].long()
    b = len(lens)
    n = max(s["table"].shape[1] * ps, budget)
    tok = torch.arange(n, device=lens.device)
    held = tok < lens[:, None]
    page = torch.where(held, s["table"][:, (tok // ps).clamp(max=s["table"].shape[1] - 1)].long(), 0)
    at = (tok % ps).expand(b, -1)
    key = s["mass"][page, :, at].transpose(1, 2)                            # (row, kv head, token)
    key = torch.where((tok >= lens[:, None] - recent)[:, None], math.inf, key).masked_fill(~held[:, None], -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    kept = torch.zeros_like(key, dtype=torch.bool).scatter_(-1, order, True) & held[:, None]
    kept = torch.where(kept, tok, n).sort(-1).values[..., :budget]          # (row, kv head, budget)
    r, g, i = ((kept < n) & (kept != tok[:budget])).nonzero(as_tuple=True)
    j = kept[r, g, i]
    src, dst = (page[r, j], at[r, j]), (page[r, i], at[r, i])
    for c in (s["k_cache"], s["v_cache"]):
        c = c.view(torch.uint8) if s["cache"] == "f8" else c
        c[dst[0], dst[1], g] = c[src[0], src[1], g]
    s["mass"][dst[0], g, dst[1]] = s["mass"][src[0], g, src[1]]
    return {"len": lens.clamp(max=budget).int(), "kept": torch.where(kept < n, kept, -1).int(), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"], "mass": s["mass"]}


_PLAIN = {"prefix": _plain_prefix, "bounds": _plain_bounds, "select": _plain_select, "sparse": _plain_sparse,
          "mass": _plain_mass, "evict": _plain_evict}


# ------------------------------------------------- the library's operators ----
def _own_run(s):
    import selective_state_space_s6_amd as m
    op = s["op"]
    if op == "prefix":
        o, lse = m.ssm_prefix_attn_decode_fwd(s["q"], s["k_cache"], s["v_cache"], s["prefix"], s["prefix_table"],
                                              s["prefix_lens"], s["table"], s["lens"], scale=s["scale"],
                                              k_scale=s["cache_scale"], v_scale=s["cache_scale"], return_lse=True)
        return {"o": o, "lse": lse}
    if op == "bounds":
        m.ssm_kv_page_bounds_update(s["k_cache"], s["bounds"], s["table"], s["len_old"], s["lens"])
        return {"bounds": s["bounds"]}
    if op == "select":
        return {"selected": m.ssm_kv_page_select_fwd(s["q"], s["bounds"], s["table"], s["lens"], page_size=s["page"],
                                                     top_k=s["top"], first=s["first"], last=s["last"])}
    if op == "sparse":
        o, lse = m.ssm_select_attn_decode_fwd(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["selected"],
                                              scale=s["scale"], k_scale=s["cache_scale"], v_scale=s["cache_scale"],
                                              return_lse=True)
        return {"o": o, "lse": lse}
    if op == "mass":
        m.ssm_kv_mass_update(s["q"], s["k_cache"], s["lse"], s["mass"], s["table"], s["starts"], s["positions"],
                             s["len_old"], s["lens"], scale=s["scale"], k_scale=s["cache_scale"])
        return {"mass": s["mass"]}
    length, kept = m.ssm_kv_evict(s["k_cache"], s["v_cache"], s["mass"], s["table"], s["lens"], budget=s["budget"],
                                  recent=s["recent"])
    return {"len": length, "kept": kept, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "mass": s["mass"]}


def run(state):
    return _own_run(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------- work ----
def work(case):
    op, ps, hk, d, c = case["op"], case["page"], case["kv_heads"], case["dim"], BYTES[case["cache"]]
    e = 4 if case["cache"] == "f32" else 2
    lens, old = _lengths(case)
    have = -(-lens // ps)
    if op == "bounds":
        first = old // ps
        pages = int(np.where(lens > old, have - first, 0).sum())
        again = int(((lens > old) & (old % ps > 0)).sum())         # pages whose bounds are read too
        return {"bytes": int((lens - old).sum()) * hk * d * c + (pages + again) * hk * 2 * d * c + 4 * pages + 8 * len(lens),
                "flops": 2 * int((lens - old).sum()) * hk * d}
    if op == "evict":
        over = lens > case["budget"]
        # of the kept tokens, those behind the first that goes
        moved = int((case["budget"] * (1 - 1 / (np.maximum(lens - case["budget"], 0) + 1)))[over].sum())
        return {"bytes": int(lens[over].sum()) * hk * 4 + moved * hk * (4 * d * c + 8) + 4 * len(lens) * hk * case["budget"]
                + 4 * int(have.sum()) + 8 * len(lens), "flops": 0}
    h = case["heads"]
    if op == "mass":
        rows = int((lens - old).sum())
        pairs = int(((lens + old + 1) * (lens - old) // 2).sum())
        live = lens[lens > old].sum()
        return {"bytes": int(live) * hk * (d * c + 8) + rows * h * (d * e + 4) + 4 * int(have.sum()) + 12 * len(lens) + 4 * rows,
                "flops": 2 * pairs * h * d}
    row = h * (2 * d * e + 4) + 4
    if op == "prefix":
        plens, of = _prefixes(case)
        used = [int(n) for p, n in enumerate(plens) if (of == p).any()]
        seen = int(lens.sum()) + int(sum(plens[p] for p in of if p >= 0))
        return {"bytes": 2 * (int(lens.sum()) + sum(used)) * hk * d * c + 4 * int(have.sum())
                + 4 * sum(-(-n // ps) for n in used) + len(lens) * (row + 4), "flops": 4 * seen * h * d}
    long = have > case["top"]
    if op == "select":
        pages = int(have[long].sum())
        return {"bytes": pages * (hk * 2 * d * c + 4) + int(long.sum()) * h * d * e + 4 * len(lens) * (1 + hk * case["top"]),
                "flops": 2 * pages * h * d}
    seen = int(np.minimum(lens, np.where(long, case["top"] * ps, lens)).sum())
    return {"bytes": 2 * seen * hk * d * c + 4 * len(lens) * hk * case["top"] + 4 * int(np.minimum(have, case["top"]).sum())
            + len(lens) * row, "flops": 4 * seen * h * d}


# --------------------------------------------------------- 64-bit answers ----
def _exact_rows(cache, pages, n, s):
    """The first n rows of a list of pages, (kv head, token, dim) in fp64."""
    x = cache.view(torch.uint8)[pages].view(cache.dtype) if s["cache"] == "f8" else cache[pages]
    return x.double().flatten(0, 1)[:n].transpose(0, 1) * s["cache_scale"]


def _exact_attend(q, k, v, scale):
    """q (kv head, group, dim) over k, v (kv head, token, dim)."""
    sc = torch.matmul(q, k.transpose(1, 2).contiguous()) * scale
    return torch.matmul(torch.softmax(sc, -1), v.contiguous()), torch.logsumexp(sc, -1)


def exact(case, seed):
    op = case["op"]
    if op == "select":
        return None    # whole numbers only
    s = prepare(case, seed)
    ps, hk, d = case["page"], case["kv_heads"], case["dim"]
    lens, old = _lengths(case)
    if op in ("prefix", "sparse"):
        h = case["heads"]
        o = torch.zeros((case["batch"], h, d), dtype=torch.float64, device="cuda")
        lse = torch.full((case["batch"], h), -math.inf, dtype=torch.float64, device="cuda")
        if op == "prefix":
            plens, of = _prefixes(case)
            kept = {p: tuple(_exact_rows(s[c], s["prefix_table"][p, :-(-int(n) // ps)].long(), int(n), s)
                             for c in ("k_cache", "v_cache")) for p, n in enumerate(plens)}
        for r, n in enumerate(lens.tolist()):
            q = s["q"][r].double().view(hk, h // hk, d)
            pages = s["table"][r, :-(-n // ps)].long()
            k, v = _exact_rows(s["k_cache"], pages, n, s), _exact_rows(s["v_cache"], pages, n, s)
            if op == "prefix" and of[r] >= 0:
                k, v = torch.cat([kept[of[r]][0], k], 1), torch.cat([kept[of[r]][1], v], 1)
            if k.shape[1] == 0:
                continue
            if op == "prefix":
                got = _exact_attend(q, k, v, s["scale"])
                o[r], lse[r] = got[0].view(h, d), got[1].view(h)
                continue
            for g in range(hk):
                mine = s["selected"][r, g]
                mine = mine[mine >= 0].long()
                j = (mine[:, None] * ps + torch.arange(ps, device="cuda")).flatten()
                j = j[j < n]
                got = _exact_attend(q[g:g + 1], k[g:g + 1, j], v[g:g + 1, j], s["scale"])
                group = slice(g * (h // hk), (g + 1) * (h // hk))
                o[r, group], lse[r, group] = got[0][0], got[1][0]
        return {"o": o, "lse": lse}
    if op == "bounds":
        b = s["bounds"].double()
        for r, n in enumerate(lens.tolist()):
            first = int(old[r])
            for i in range(first // ps, -(-n // ps) if n > first else 0):
                p = int(s["table"][r, i])
                lo, hi = max(first - i * ps, 0), min(n - i * ps, ps)
                k = s["k_cache"][p, lo:hi].double()
                if lo > 0:
                    k = torch.cat([k, b[p].transpose(0, 1)])
                b[p, :, 0], b[p, :, 1] = k.min(0).values, k.max(0).values
            if r * max(1, case["grow"] // ps) > 20000:
                return None
        return {"bounds": b}
    if op == "mass":
        h = case["heads"]
        mass = s["mass"].double()
        starts = np.concatenate([[0], np.cumsum(lens - old)])
        for r, n in enumerate(lens.tolist()):
            if n == 0:
                continue
            pages = s["table"][r, :-(-n // ps)].long()
            k = _exact_rows(s["k_cache"], pages, n, s).transpose(1, 2).contiguous()
            sums = torch.zeros((hk, n), dtype=torch.float64, device="cuda")
            for a in range(int(starts[r]), int(starts[r + 1]), 256):
                t = torch.arange(a, min(a + 256, int(starts[r + 1])), device="cuda")
                sc = torch.matmul(s["q"][t].double().view(len(t), hk, h // hk, d).transpose(0, 1).flatten(1, 2), k) * s["scale"]
                w = torch.exp(sc.view(hk, len(t), h // hk, n) - s["lse"][t].double().view(len(t), hk, h // hk).transpose(0, 1)[..., None])
                sees = torch.arange(n, device="cuda") <= s["positions"][t].long()[:, None]
                sums += (w * sees[None, :, None]).sum((1, 2))
            j = torch.arange(n, device="cuda")
            was = mass[pages[j // ps], :, j % ps] * (j < int(old[r]))[:, None]
            mass[pages[j // ps], :, j % ps] = was + sums.T
        return {"mass": mass}
    # kept tokens are whole numbers, and moved rows the values that were there
    k_cache, v_cache, mass = (s[c].double() for c in ("k_cache", "v_cache", "mass"))
    for r, n in enumerate(lens.tolist()):
        if n <= case["budget"]:
            continue
        pages = s["table"][r].long()
        for g in range(hk):
            j = torch.arange(n, device="cuda")
            key = mass[pages[j // ps], g, j % ps].cpu().numpy()
            early = n - case["recent"]
            best = np.lexsort((np.arange(early), -key[:early]))[:case["budget"] - case["recent"]]
            j = torch.from_numpy(np.concatenate([np.sort(best), np.arange(early, n)])).cuda()
            i = torch.arange(case["budget"], device="cuda")
            for c in (k_cache, v_cache):
                c[pages[i // ps], i % ps, g] = c[pages[j // ps], j % ps, g]
            mass[pages[i // ps], g, i % ps] = mass[pages[j // ps], g, j % ps]
    return {"len": None, "kept": None, "k_cache": k_cache, "v_cache": v_cache, "mass": mass}
