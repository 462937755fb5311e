"""Measured cases of the operators around attention over a paged key-value cache.

Four operators: the cache's page bookkeeping (``pages``), RMS norm and position rotation of
q and k heads with its gradients (``rope``, ``rope_bwd``), the same pass writing k and v into
the cache (``rope_cache``), and attention of one new token over the cache (``attn``).

``own`` picks what ``run`` does: the plain torch form, or the library's entry points.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f8": 1}
CACHE_SCALE = 0.03125     # an 8-bit cache holds k / CACHE_SCALE, v / CACHE_SCALE


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one decode step of a full batch: every request one token longer, each 16th one done
        {"name": "pages decode 256", "op": "pages", "batch": 256, "old": 4096, "grow": 1, "page": 16,
         "done_every": 16, "tight": False},
        # a step that admits prompts of very different lengths, more than there are pages for
        {"name": "pages prompts 512", "op": "pages", "batch": 512, "old": 0, "grow": 2048, "page": 16,
         "done_every": 0, "tight": True},
        # a training batch of 4 x 4096 tokens, grouped heads
        {"name": "rope train bf16", "op": "rope", "tokens": 16384, "heads": 16, "kv_heads": 4, "dim": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "norm": True},
        # an odd number of tokens, a partly rotated head of odd size, neighbouring pairs, fp32
        {"name": "rope odd f32", "op": "rope", "tokens": 1021, "heads": 6, "kv_heads": 3, "dim": 72, "rot": 24,
         "dtype": "f32", "interleaved": True, "norm": True},
        {"name": "rope bwd bf16", "op": "rope_bwd", "tokens": 16384, "heads": 16, "kv_heads": 4, "dim": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "norm": True},
        {"name": "rope bwd odd f32", "op": "rope_bwd", "tokens": 1021, "heads": 6, "kv_heads": 3, "dim": 72, "rot": 24,
         "dtype": "f32", "interleaved": True, "norm": True},
        # a decode step: one token of each of 64 requests into the cache
        {"name": "cache decode 64", "op": "rope_cache", "tokens": 64, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "dtype": "bf16", "cache": "bf16", "page": 16, "layout": "nhd", "interleaved": False, "norm": True},
        # a prompt chunk into an 8-bit cache that keeps each head's tokens of a page together
        {"name": "cache prompt f8", "op": "rope_cache", "tokens": 8192, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 64,
         "dtype": "bf16", "cache": "f8", "page": 64, "layout": "hnd", "interleaved": False, "norm": True},
        # one request alone: latency
        {"name": "attn one", "op": "attn", "batch": 1, "len": 2047, "ragged": False, "heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "cache": "bf16", "page": 16, "layout": "nhd", "window": 0},
        # a batch in the middle of its answers: all lengths up to 8192, an idle place in it
        {"name": "attn batch ragged", "op": "attn", "batch": 64, "len": 8192, "ragged": True, "heads": 32, "kv_heads": 8,
         "dim": 128, "dtype": "bf16", "cache": "bf16", "page": 16, "layout": "nhd", "window": 0},
        # long contexts in an 8-bit cache
        {"name": "attn long f8", "op": "attn", "batch": 16, "len": 65536, "ragged": False, "heads": 64, "kv_heads": 8,
         "dim": 128, "dtype": "bf16", "cache": "f8", "page": 64, "layout": "hnd", "window": 0},
        # one shared wide key-value head in fp32 with a sliding window
        {"name": "attn shared f32", "op": "attn", "batch": 48, "len": 5000, "ragged": True, "heads": 5, "kv_heads": 1,
         "dim": 256, "dtype": "f32", "cache": "f32", "page": 24, "layout": "nhd", "window": 4001},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "rope", "rope_bwd", "rope_cache", "attn", "attn"])
    if op == "pages":
        grow = rng.choice([1, 1, _log(rng, 2, 2048)])
        return {"op": op, "batch": _log(rng, 1, 512), "old": rng.choice([0, _log(rng, 1, 16384)]), "grow": grow,
                "page": rng.choice([1, 8, 16, 24, 64, 256]) if grow < 256 else rng.choice([16, 24, 64, 256]),
                "done_every": rng.choice([0, 3, 16]), "tight": rng.random() < 0.4}
    kv = rng.choice([1, 2, 3, 4, 8])
    case = {"op": op, "heads": kv * rng.choice([1, 2, 3, 4, 5, 8]), "kv_heads": kv}
    if op == "attn":
        case.update(dim=rng.choice([64, 80, 96, 128, 128, 192, 256]), page=rng.choice([1, 8, 16, 16, 24, 64, 128]),
                    layout=rng.choice(["nhd", "hnd"]), window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]),
                    ragged=rng.random() < 0.7)
        case["dtype"], case["cache"] = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "f8"), ("f32", "f32")])
        case["batch"] = _log(rng, 1, 256)
        room = 4e8 / (case["batch"] * kv * case["dim"])
        case["len"] = max(1, min(_log(rng, 1, 131072), int(room)))
        return case
    case["dim"] = rng.choice([64, 72, 80, 96, 128, 128, 256])
    case["rot"] = rng.choice([case["dim"], case["dim"] // 16 * 8, 24])
    case["dtype"] = rng.choice(["bf16", "bf16", "f32"])
    case["interleaved"], case["norm"] = rng.random() < 0.4, rng.random() < 0.8
    case["tokens"] = min(_log(rng, 1, 16384), int(16384 * 20 * 128 / ((case["heads"] + 2 * kv) * case["dim"])))
    if op == "rope_cache":
        case["cache"] = rng.choice(["bf16", "f8"]) if case["dtype"] == "bf16" else "f32"
        if case["cache"] == "f8" and case["dim"] % 16:
            case["dim"], case["rot"] = 96, 48
        case.update(page=rng.choice([1, 8, 16, 24, 64]), layout=rng.choice(["nhd", "hnd"]))
    return case


def _lengths(case):
    """The requests' cached tokens: all `len`, or spread over 1..len with one idle place."""
    n, top = case["batch"], case["len"]
    if not case["ragged"]:
        return np.full(n, top, dtype=np.int64)
    part = np.modf(0.5 + 0.6180339887498949 * np.arange(n))[0]
    got = 1 + (part * (top - 1)).astype(np.int64)
    if n >= 4:
        got[3] = 0
    return got


def _page_lengths(case):
    """(tokens held, tokens to hold) of each request of a `pages` case."""
    n = np.arange(case["batch"])
    part = np.modf(0.5 + 0.6180339887498949 * n)[0]
    held = (case["old"] * (0.5 + part)).astype(np.int64)
    grow = np.ones_like(held) if case["grow"] == 1 else 1 + (part * (case["grow"] - 1)).astype(np.int64)
    hold = held + grow
    if case["done_every"]:
        hold[n % case["done_every"] == case["done_every"] - 1] = 0
    return held, hold


# ----------------------------------------------------------------- inputs ----
def _cache(case, pages, g, fill):
    """A (pages, page, kv_heads, dim) view of a cache in the case's layout."""
    dtype, hk, d, ps = DTYPES[case["cache"]], case["kv_heads"], case["dim"], case["page"]
    shape = (pages, ps, hk, d) if case["layout"] == "nhd" else (pages, hk, ps, d)
    if fill:
        kind = torch.float32 if dtype == torch.float32 else torch.bfloat16
        c = torch.randn(shape, generator=g, device="cuda", dtype=kind)
        c = c.div_(CACHE_SCALE).to(dtype) if case["cache"] == "f8" else c
    else:
        c = torch.zeros(shape, device="cuda", dtype=torch.uint8).view(dtype) if case["cache"] == "f8" else \
            torch.zeros(shape, device="cuda", dtype=dtype)
    return c if case["layout"] == "nhd" else c.permute(0, 2, 1, 3)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 32))
    s = dict(case)

    def ints(a, dtype=torch.int32):
        return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)

    if case["op"] == "pages":
        held, hold = _page_lengths(case)
        ps = case["page"]
        have, want = -(-held // ps), -(-hold // ps)
        cols = int(max(have.max(), want.max())) + 1
        need = int(np.maximum(want - have, 0).sum())
        free = max(1, int(need * 0.75)) if case["tight"] else need + max(8, need // 4)
        total = int(have.sum()) + free
        order = rs.permutation(total)
        table = np.zeros((case["batch"], cols), dtype=np.int64)
        table[np.arange(cols)[None] < have[:, None]] = order[:int(have.sum())]
        head = int(rs.randint(total))
        ring = np.zeros(total, dtype=np.int64)
        ring[(head + np.arange(free)) % total] = order[int(have.sum()):]
        s.update(len_old=ints(held), len_new=ints(hold), table=ints(table), free_ring=ints(ring),
                 ring=ints(np.array([head, free])), n_tokens=int(np.maximum(hold - held, 0).sum()) + 5)
        return s

    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "attn":
        lens = _lengths(case)
        ps = case["page"]
        have = -(-lens // ps)
        cols, total = max(1, int(-(-case["len"] // ps))), int(have.sum()) + 3
        table = np.full((case["batch"], cols), -1, dtype=np.int64)
        table[np.arange(cols)[None] < have[:, None]] = rs.permutation(total)[:int(have.sum())]
        s.update(q=torch.randn((case["batch"], h, d), generator=g, device="cuda", dtype=dtype),
                 k_cache=_cache(case, total, g, True), v_cache=_cache(case, total, g, True),
                 table=ints(table), lens=ints(lens), scale=d ** -0.5,
                 cache_scale=CACHE_SCALE if case["cache"] == "f8" else 1.0)
        return s

    t = case["tokens"]
    # q, k, v as one projection gives them: slices of a row of all heads
    qkv = torch.randn((t, (h + 2 * hk) * d), generator=g, device="cuda", dtype=dtype)
    s["q"] = qkv[:, :h * d].view(t, h, d)
    s["k"] = qkv[:, h * d:(h + hk) * d].view(t, hk, d)
    s["v"] = qkv[:, (h + hk) * d:].view(t, hk, d)
    s["wq"], s["wk"] = ((1.0 + 0.1 * torch.randn((d,), generator=g, device="cuda")) if case["norm"] else None
                        for _ in range(2))
    half = case["rot"] // 2
    s["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
    s["positions"] = ints(rs.randint(0, 131072) + np.arange(t))
    if case["op"] == "rope_bwd":
        s["dq_out"] = torch.randn((t, h, d), generator=g, device="cuda", dtype=dtype)
        s["dk_out"] = torch.randn((t, hk, d), generator=g, device="cuda", dtype=dtype)
    if case["op"] == "rope_cache":
        ps = case["page"]
        total = -(-t // ps) + 4
        s["slots"] = ints(rs.permutation(total * ps)[:t], torch.int64)
        s["k_cache"], s["v_cache"] = _cache(case, total, g, False), _cache(case, total, g, False)
        s["cache_scale"] = CACHE_SCALE if case["cache"] == "f8" else 1.0
    return s


# ------------------------------------------------------------ plain forms ----
def _plain_pages(s):
    ps, dev = s["page"], s["len_old"].device
    old, new = s["len_old"].long().clamp(min=0), s["len_new"].long().clamp(min=0)
    table, ring = s["table"], s["free_ring"]
    cols, total = table.shape[1], ring.shape[0]
    head, free = s["ring"][0].long(), s["ring"][1].long()
    have, want = (old + ps - 1) // ps, (new + ps - 1) // ps
    long = want > cols
    need = torch.where(long, 0, (want - have).clamp(min=0))
    refused = long | ((need > 0) & (need.cumsum(0) > free))
    take = torch.where(refused, 0, need)
    take_at = take.cumsum(0) - take
    give = (have - want).clamp(min=0)
    give_to = give.cumsum(0)
    grow = (new - old).clamp(min=0)
    ends = grow.cumsum(0)
    starts = torch.cat([ends.new_zeros(1), ends])
    # released pages go behind the ring's last entry
    i = (torch.arange(total, device=dev) - head - free) % total
    r = torch.searchsorted(give_to, i, right=True).clamp(max=len(old) - 1)
    c = (want[r] + i - (give_to - give)[r]).clamp(0, cols - 1)
    ring_new = torch.where(i < give_to[-1], table[r, c], ring)
    # taken pages come from its head
    c = torch.arange(cols, device=dev)[None]
    at = (head + take_at[:, None] + c - have[:, None]) % total
    fresh = (c >= have[:, None]) & (c < (have + take)[:, None])
    table_new = torch.where(fresh, ring[at], table)
    t = torch.arange(s["n_tokens"], device=dev)
    r = torch.searchsorted(ends, t, right=True)
    inside = r < len(old)
    r = r.clamp(max=len(old) - 1)
    pos = old[r] + t - starts[r]
    page = table_new[r, (pos // ps).clamp(max=cols - 1)].long()
    slot = torch.where(inside & ~refused[r], page * ps + pos % ps, -1)
    taken = take.sum()
    table.copy_(table_new)
    ring.copy_(ring_new)
    return {"block_table": table, "free_ring": ring,
            "ring": torch.stack([(head + taken) % total, free - taken + give_to[-1]]).int(),
            "len": torch.where(refused, old, new).int(), "starts": starts.int(),
            "request": torch.where(inside, r, -1).int(), "positions": torch.where(inside, pos, -1).int(),
            "slots": slot, "denied": refused.sum().int().reshape(1)}


def _cos_sin(s):
    ang = s["positions"].double()[:, None] * s["inv_freq"].double()
    return ang.cos().float()[:, None], ang.sin().float()[:, None]


def _rotate(x, cos, sin, rot, interleaved):
    """The first `rot` values of each head, turned by the angles in pairs."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_rope_one(x, w, s, cos, sin):
    y = x.float()
    if s["norm"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
    return _rotate(y, cos, sin, s["rot"], s["interleaved"])


def _plain_rope(s):
    cos, sin = _cos_sin(s)
    return {n: _plain_rope_one(s[n], s["w" + n], s, cos, sin).to(s[n].dtype) for n in ("q", "k")}


def _plain_rope_bwd_one(x, w, dy, s, cos, sin):
    g = _rotate(dy.float(), cos, -sin, s["rot"], s["interleaved"])
    if not s["norm"]:
        return g.to(x.dtype), None
    x32 = x.float()
    r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    n = x32 * r
    wg = g * w
    dx = r * (wg - n * (wg * n).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * n).double().sum((0, 1)).float()


def _plain_rope_bwd(s):
    cos, sin = _cos_sin(s)
    dq, dwq = _plain_rope_bwd_one(s["q"], s["wq"], s["dq_out"], s, cos, sin)
    dk, dwk = _plain_rope_bwd_one(s["k"], s["wk"], s["dk_out"], s, cos, sin)
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _plain_store(cache, x, s):
    page, at = s["slots"] // s["page"], s["slots"] % s["page"]
    if cache.dtype == torch.float8_e4m3fn:
        x = (x.float() / s["cache_scale"]).clamp(-448.0, 448.0).to(cache.dtype)
        cache.view(torch.uint8)[page, at] = x.view(torch.uint8)
    else:
        cache[page, at] = x.to(cache.dtype)


def _plain_rope_cache(s):
    cos, sin = _cos_sin(s)
    q = _plain_rope_one(s["q"], s["wq"], s, cos, sin).to(s["q"].dtype)
    _plain_store(s["k_cache"], _plain_rope_one(s["k"], s["wk"], s, cos, sin), s)
    _plain_store(s["v_cache"], s["v"], s)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(cache, page, at, valid, scale):
    if cache.dtype == torch.float8_e4m3fn:
        x = cache.view(torch.uint8)[page, at].view(cache.dtype).float() * scale
    else:
        x = cache[page, at].float()
    return x.masked_fill_(~valid[..., None, None], 0.0)


def _plain_attn(s):
    q, ps, hk = s["q"], s["page"], s["kv_heads"]
    b, h, d = q.shape
    tok = torch.arange(s["table"].shape[1] * ps, device=q.device)
    lens = s["lens"].long()[:, None]
    valid = tok < lens
    if s["window"] > 0:
        valid = valid & (tok >= lens - s["window"])
    page = torch.where(valid, s["table"][:, tok // ps].long(), 0)
    at = (tok % ps).expand(b, -1)
    k = _gathered(s["k_cache"], page, at, valid, s["cache_scale"])
    sc = torch.matmul(q.float().view(b, hk, h // hk, d), k.permute(0, 2, 3, 1)) * s["scale"]
    del k
    sc = sc.masked_fill(~valid[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(sc - top)
    mass = p.sum(-1, keepdim=True)
    v = _gathered(s["v_cache"], page, at, valid, s["cache_scale"])
    o = torch.matmul(p, v.transpose(1, 2)) / torch.where(mass > 0, mass, 1.0)
    return {"o": o.view(b, h, d).to(q.dtype), "lse": (top + torch.log(mass)).view(b, h)}


_PLAIN = {"pages": _plain_pages, "rope": _plain_rope, "rope_bwd": _plain_rope_bwd, "rope_cache": _plain_rope_cache,
          "attn": _plain_attn}


# ------------------------------------------------- the library's operators ----
def _flags(s, m):
    return (m.SSM_ROPE_INTERLEAVED if s["interleaved"] else 0) | (0 if s["norm"] else m.SSM_QK_NO_NORM)


def _own_run(s):
    import selective_state_space_s6_amd as m
    op = s["op"]
    if op == "pages":
        got = m.ssm_kv_pages_step(s["len_old"], s["len_new"], s["table"], s["free_ring"], s["ring"],
                                  page_size=s["page"], n_tokens=s["n_tokens"])
        return {"block_table": s["table"], "free_ring": s["free_ring"], "ring": got["ring"], "len": got["len"],
                "starts": got["starts"], "request": got["request"], "positions": got["positions"],
                "slots": got["slots"], "denied": got["denied"]}
    if op == "rope":
        q, k = m.ssm_qk_norm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["positions"], eps=EPS,
                                      flags=_flags(s, m))
        return {"q": q, "k": k}
    if op == "rope_bwd":
        got = m.ssm_qk_norm_rope_bwd(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["positions"], s["dq_out"],
                                     s["dk_out"], eps=EPS, flags=_flags(s, m))
        return {n: got[n] for n in ("dq", "dk", "dwq", "dwk")}
    if op == "rope_cache":
        q = m.ssm_qk_norm_rope_cache_fwd(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["inv_freq"], s["positions"],
                                         s["slots"], s["k_cache"], s["v_cache"], eps=EPS, k_scale=s["cache_scale"],
                                         v_scale=s["cache_scale"], flags=_flags(s, m))
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    o, lse = m.ssm_paged_attn_decode_fwd(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], scale=s["scale"],
                                         window=s["window"], k_scale=s["cache_scale"], v_scale=s["cache_scale"],
                                         return_lse=True)
    return {"o": o, "lse": lse}


def run(state):
    return _own_run(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------- work ----
def work(case):
    op = case["op"]
    if op == "pages":
        held, hold = _page_lengths(case)
        ps = case["page"]
        have, want = -(-held // ps), -(-hold // ps)
        tokens = int(np.maximum(hold - held, 0).sum()) + 5
        moved = int(np.abs(want - have).sum())
        # two lengths in, length and start out; 16 B a token; a page id read and written where it moves
        return {"bytes": 16 * case["batch"] + 16 * tokens + 8 * moved, "flops": 0}
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    e = BYTES[case["dtype"]]
    if op == "attn":
        lens = _lengths(case)
        seen = int((np.minimum(lens, case["window"]) if case["window"] else lens).sum())
        c = BYTES[case["cache"]]
        return {"bytes": 2 * seen * hk * d * c + 4 * (-(-seen // case["page"])) + 4 * len(lens)
                + len(lens) * h * (2 * d * e + 4), "flops": 4 * seen * h * d}
    t = case["tokens"]
    small = 4 * t + 2 * case["rot"] + 8 * d
    if op == "rope":
        return {"bytes": 2 * t * (h + hk) * d * e + small, "flops": 8 * t * (h + hk) * d}
    if op == "rope_bwd":
        return {"bytes": (3 if case["norm"] else 2) * t * (h + hk) * d * e + small, "flops": 16 * t * (h + hk) * d}
    return {"bytes": t * (h + 2 * hk) * d * e + t * h * d * e + 2 * t * hk * d * BYTES[case["cache"]] + 8 * t + small,
            "flops": 8 * t * (h + hk) * d}


# --------------------------------------------------------- 64-bit answers ----
def _exact_head(x, w, s):
    """norm and rotation of heads x (tokens, heads, dim), as complex turns, in fp64."""
    if s["norm"]:
        x = w.double() * x / torch.sqrt(torch.einsum("thd,thd->th", x, x)[..., None] / x.shape[-1] + EPS)
    half = s["rot"] // 2
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       torch.outer(s["positions"].double(), s["inv_freq"].double()))[:, None, :]
    head, rest = x[..., :s["rot"]], x[..., s["rot"]:]
    pairs = head.unflatten(-1, (half, 2)) if s["interleaved"] else head.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * turn)
    z = z if s["interleaved"] else z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), rest], dim=-1)


def exact(case, seed):
    if case["op"] == "pages":
        return None    # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "attn":
        b, h, d = s["q"].shape
        hk, ps = case["kv_heads"], case["page"]
        o = torch.zeros((b, h, d), dtype=torch.float64, device="cuda")
        lse = torch.full((b, h), -math.inf, dtype=torch.float64, device="cuda")
        f8 = case["cache"] == "f8"

        def rows(cache, pages, first, last):
            x = (cache.view(torch.uint8)[pages].view(cache.dtype) if f8 else cache[pages]).double()
            return x.reshape(-1, hk, d)[first:last] * s["cache_scale"]

        for r, n in enumerate(_lengths(case).tolist()):
            first = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                continue
            from_page = first // ps
            pages = s["table"][r, from_page:-(-n // ps)].long()
            first, last = first - from_page * ps, n - from_page * ps
            k = rows(s["k_cache"], pages, first, last)
            q = s["q"][r].double().view(hk, h // hk, d)
            score = torch.bmm(q, k.permute(1, 2, 0).contiguous()) * s["scale"]
            lse[r] = torch.logsumexp(score, -1).view(-1)
            v = rows(s["v_cache"], pages, first, last)
            o[r] = torch.bmm(torch.softmax(score, -1), v.transpose(0, 1).contiguous()).view(h, d)
        return {"o": o, "lse": lse}
    if case["op"] == "rope_bwd":
        got = {}
        for n in ("q", "k"):
            x = s[n].double().clone().requires_grad_(True)
            w = s["w" + n].double().clone().requires_grad_(True) if case["norm"] else None
            grads = torch.autograd.grad(_exact_head(x, w, s), [x] + ([w] if case["norm"] else []),
                                        s["d" + n + "_out"].double())
            got["d" + n], got["dw" + n] = grads[0], grads[1] if case["norm"] else None
        return got
    q, k = (_exact_head(s[n].double(), s["w" + n], s) for n in ("q", "k"))
    if case["op"] == "rope":
        return {"q": q, "k": k}
    if case["cache"] == "f8":
        return {"q": q, "k_cache": None, "v_cache": None}
    kc, vc = (torch.zeros(s["k_cache"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    where = (s["slots"] // case["page"], s["slots"] % case["page"])
    kc[where], vc[where] = k, s["v"].double()
    return {"q": q, "k_cache": kc, "v_cache": vc}
