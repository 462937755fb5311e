"""include/ssm_longctx.h without a GPU: every declared symbol is exported, workspace sizes, and
every argument check returns its code and message before any HIP call (the addresses are
never dereferenced on these paths); the binding's own checks of dtype, shape, stride and
device."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssm_longctx.h")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
INF = float("inf")


@pytest.fixture(scope="module")
def m():
    import selective_state_space_s6_amd as m
    return m


@pytest.fixture(scope="module")
def lib(m):
    L = ctypes.CDLL(m.LIB_PATH)
    I, P, Z, F, D = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float, ctypes.c_int
    L.ssm_last_error.restype = ctypes.c_char_p
    L.ssm_prefix_attn_decode_fwd.argtypes = [P] * 10 + [I] * 16 + [F] * 3 + [D, D, P, Z, P]
    L.ssm_kv_page_bounds_update.argtypes = [P] * 5 + [I] * 10 + [D, P]
    L.ssm_kv_page_select_fwd.argtypes = [P] * 5 + [I] * 13 + [D, D, P, Z, P]
    L.ssm_select_attn_decode_fwd.argtypes = [P] * 8 + [I] * 14 + [F] * 3 + [D, D, P, Z, P]
    L.ssm_kv_mass_update.argtypes = [P] * 9 + [I] * 14 + [F, F, D, D, P]
    L.ssm_kv_evict.argtypes = [P] * 7 + [I] * 12 + [D, P]
    for n, k in (("prefix_attn_decode_fwd", 7), ("kv_page_select_fwd", 4), ("select_attn_decode_fwd", 7)):
        f = getattr(L, f"ssm_{n}_workspace_size")
        f.argtypes, f.restype = [I] * k, Z
    return L


def _p(i):
    return ctypes.c_void_p(0x100000 * (i + 1))


def _table(lib, fn, order, base, cases):
    for kw, code, word in cases:
        a = dict(base, **kw)
        assert set(a) == set(order)
        assert getattr(lib, fn)(*(a[n] for n in order)) == code, (fn, kw, lib.ssm_last_error())
        err = lib.ssm_last_error().decode()
        if code != OK:
            assert word in err and err.startswith(fn), (kw, err)


def test_every_declared_symbol_is_exported(m, lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(ssm_\w+)\s*\(", text))
    assert names == {"ssm_prefix_attn_decode_fwd", "ssm_prefix_attn_decode_fwd_workspace_size", "ssm_kv_page_bounds_update",
                     "ssm_kv_page_select_fwd", "ssm_kv_page_select_fwd_workspace_size", "ssm_select_attn_decode_fwd",
                     "ssm_select_attn_decode_fwd_workspace_size", "ssm_kv_mass_update", "ssm_kv_evict"}
    for n in names:
        assert hasattr(lib, n) and n in m.__all__ and callable(getattr(m, n))


CACHE = ["n_pages", "page_size"]
STRIDES = ["c_sp", "c_st", "c_sh"]
SIZES = dict(n_pages=32, page_size=16, c_sp=2048, c_st=128, c_sh=64)
# what every entry point over a paged cache refuses
PAGED = [
    (dict(batch=-1), INVALID, "must be >= 0"), (dict(n_kv=0), INVALID, "n_kv_heads"), (dict(d=0), INVALID, "headdim"),
    (dict(d=264), UNSUPPORTED, "headdim 264 > 256"), (dict(d=60), UNSUPPORTED, "multiple of 8"),
    (dict(d=72, kv=2), UNSUPPORTED, "multiple of 16"), (dict(max_pages=0, table_stride=0), INVALID, "max_pages"),
    (dict(table_stride=7), INVALID, "table_stride 7 < max_pages 8"), (dict(n_pages=0), INVALID, "n_pages"),
    (dict(page_size=0), INVALID, "page_size"), (dict(n_pages=1 << 30), UNSUPPORTED, "2^31"),
    (dict(max_pages=1 << 27, table_stride=1 << 27), UNSUPPORTED, "too large"),
]
STRIDED = [
    (dict(c_sp=-1), INVALID, "strides must be >= 0"), (dict(c_st=132), UNSUPPORTED, "multiple of 16 bytes"),
    (dict(c_sp=1 << 36), UNSUPPORTED, "2^36"),
]
HEADS = [
    (dict(H=9), INVALID, "not a multiple"), (dict(H=0), INVALID, "n_heads"), (dict(dtype=2), INVALID, "dtype 2"),
    (dict(dtype=0), UNSUPPORTED, "does not go with"), (dict(kv=3), UNSUPPORTED, "does not go with"),
    (dict(q_sr=516), UNSUPPORTED, "stride of q"), (dict(q_sh=68), UNSUPPORTED, "stride of q"),
    (dict(q=ctypes.c_void_p(0x100008)), UNSUPPORTED, "q is not 16-byte"), (dict(q=None), INVALID, "q is NULL"),
]
SCALES = [(dict(scale=INF), INVALID, "scale must be finite"), (dict(k_scale=0.0, kv=2), INVALID, "k_scale")]

PREFIX = ["q", "k", "v", "prefix", "prefix_table", "prefix_lens", "table", "lens", "o", "lse", "batch", "H", "n_kv", "d", "n_prefixes",
          "max_prefix_pages", "prefix_stride", "max_pages", "table_stride"] + CACHE + ["q_sr", "q_sh"] + STRIDES + [
          "scale", "k_scale", "v_scale", "dtype", "kv", "ws", "ws_bytes", "stream"]


def _base(order, n, **kw):
    b = {x: _p(i) for i, x in enumerate(order[:n])}
    b.update(SIZES)
    b.update(batch=4, H=8, n_kv=2, d=64, max_pages=8, table_stride=8, q_sr=512, q_sh=64, scale=0.125, k_scale=1.0, v_scale=1.0,
             dtype=1, kv=1, stream=None, **kw)
    return {x: b[x] for x in order}


def _aliases(base, outs, ins):
    return [({o: base[i]}, INVALID, f"aliases {n}") for o in outs for i, n in ins.items()]


def test_prefix_checks(lib):
    need = lib.ssm_prefix_attn_decode_fwd_workspace_size(4, 8, 2, 64, 16, 8, 16)
    assert need > 0 and lib.ssm_prefix_attn_decode_fwd_workspace_size(4, 9, 2, 64, 16, 8, 16) == 0
    base = _base(PREFIX, 10, n_prefixes=3, max_prefix_pages=16, prefix_stride=16, ws=_p(20), ws_bytes=need)
    _table(lib, "ssm_prefix_attn_decode_fwd", PREFIX, base, PAGED + STRIDED + HEADS + SCALES + [
        (dict(n_prefixes=0), INVALID, "n_prefixes"), (dict(max_prefix_pages=0), INVALID, "max_prefix_pages"),
        (dict(prefix_stride=15), INVALID, "prefix_stride 15"), (dict(max_prefix_pages=1 << 27, prefix_stride=1 << 27), UNSUPPORTED, "too large"),
        (dict(batch=1 << 21), UNSUPPORTED, "too large"), (dict(v_scale=-1.0, kv=2), INVALID, "v_scale"),
        (dict(prefix=None), INVALID, "prefix is NULL"), (dict(prefix_lens=None), INVALID, "prefix_lens"), (dict(o=None), INVALID, "o is NULL"),
        (dict(v=ctypes.c_void_p(0x200008)), UNSUPPORTED, "v_cache is not 16"), (dict(o=ctypes.c_void_p(0x200008)), UNSUPPORTED, "o is not 16"),
        (dict(ws=None), WORKSPACE, "workspace"), (dict(ws_bytes=need - 1), WORKSPACE, "workspace"), (dict(lse=base["o"]), INVALID, "aliases"),
        (dict(ws=base["o"]), INVALID, "aliases"), (dict(batch=0, q=None), OK, ""),
    ] + _aliases(base, ["o", "lse", "ws"], {"q": "q", "k": "k_cache", "v": "v_cache", "prefix": "prefix", "prefix_table": "prefix_table",
                                            "prefix_lens": "prefix_lens", "table": "block_table", "lens": "lens"}))


def test_prefixes_too_long_together(lib):
    """What a block may walk is counted in 32 bits: 64 prefixes, or all of them, in tiles of 16 tokens."""
    base = _base(PREFIX, 10, n_prefixes=3, max_prefix_pages=16, prefix_stride=1 << 26, ws=None, ws_bytes=0)
    long = lambda n, tokens: dict(n_prefixes=n, max_prefix_pages=tokens // 16)  # noqa: E731
    _table(lib, "ssm_prefix_attn_decode_fwd", PREFIX, base, [
        (long(32, 1 << 30), UNSUPPORTED, "too long together"), (long(31, 1 << 30), WORKSPACE, "workspace"),
        (long(64, 1 << 29), UNSUPPORTED, "too long together"), (long(64, (1 << 29) - 16), WORKSPACE, "workspace"),
        (long(1 << 20, 1 << 29), UNSUPPORTED, "too long together"), (long(1 << 20, (1 << 29) - 16), WORKSPACE, "workspace"),
        (dict(n_prefixes=32, page_size=1 << 20, n_pages=8, c_st=64, c_sh=64, c_sp=64, max_prefix_pages=1 << 10), UNSUPPORTED, "too long together"),
        (dict(n_prefixes=1 << 31), UNSUPPORTED, "too large"),
    ])


BOUNDS = ["k", "bounds", "table", "len_old", "lens", "batch", "n_kv", "d", "max_pages", "table_stride"] + CACHE + STRIDES + ["kv", "stream"]


def test_bounds_checks(lib):
    base = _base(BOUNDS, 5)
    _table(lib, "ssm_kv_page_bounds_update", BOUNDS, base, PAGED + STRIDED + [
        (dict(kv=3), INVALID, "kv_dtype 3"), (dict(batch=4097), UNSUPPORTED, "batch 4097"), (dict(k=None), INVALID, "k_cache is NULL"),
        (dict(bounds=None), INVALID, "bounds is NULL"), (dict(len_old=None), INVALID, "len_old"), (dict(lens=None), INVALID, "lens"),
        (dict(bounds=ctypes.c_void_p(0x200008)), UNSUPPORTED, "bounds is not 16"), (dict(batch=0, k=None), OK, ""),
    ] + _aliases(base, ["bounds"], {"k": "k_cache", "table": "block_table", "len_old": "len_old", "lens": "lens"}))


SELECT = ["q", "bounds", "table", "lens", "selected", "batch", "H", "n_kv", "d", "max_pages", "table_stride"] + CACHE + [
          "top_k", "first", "last", "q_sr", "q_sh", "dtype", "kv", "ws", "ws_bytes", "stream"]


def test_select_checks(lib):
    need = lib.ssm_kv_page_select_fwd_workspace_size(4, 2, 8, 4)
    assert need > 0 and lib.ssm_kv_page_select_fwd_workspace_size(4, 2, 8, 8) == 0
    base = _base(SELECT, 5, top_k=4, first=1, last=1, ws=_p(20), ws_bytes=need)
    _table(lib, "ssm_kv_page_select_fwd", SELECT, base, PAGED + HEADS + [
        (dict(top_k=0, first=0, last=0), INVALID, "top_k"), (dict(first=-1), INVALID, "first"), (dict(last=-1), INVALID, "last"),
        (dict(first=3, last=2), INVALID, "first 3 + last 2 > top_k 4"), (dict(last=(1 << 63) - 1), INVALID, "last"),
        (dict(top_k=(1 << 20) + 1), UNSUPPORTED, "top_k"), (dict(bounds=None), INVALID, "bounds is NULL"),
        (dict(selected=None), INVALID, "selected is NULL"), (dict(ws=None), WORKSPACE, "workspace"),
        (dict(ws_bytes=need - 1), WORKSPACE, "workspace"), (dict(ws=base["selected"]), INVALID, "aliases"), (dict(batch=0, q=None), OK, ""),
    ] + _aliases(base, ["selected", "ws"], {"q": "q", "bounds": "bounds", "table": "block_table", "lens": "lens"}))


SPARSE = ["q", "k", "v", "table", "lens", "selected", "o", "lse", "batch", "H", "n_kv", "d", "max_pages", "table_stride"] + CACHE + [
          "top_k", "q_sr", "q_sh"] + STRIDES + ["scale", "k_scale", "v_scale", "dtype", "kv", "ws", "ws_bytes", "stream"]


def test_select_attn_checks(lib):
    need = lib.ssm_select_attn_decode_fwd_workspace_size(4, 8, 2, 64, 8, 16, 4)
    assert 0 < need <= lib.ssm_select_attn_decode_fwd_workspace_size(4, 8, 2, 64, 8, 16, 100)
    base = _base(SPARSE, 8, top_k=4, ws=_p(20), ws_bytes=need)
    _table(lib, "ssm_select_attn_decode_fwd", SPARSE, base, PAGED + STRIDED + HEADS + SCALES + [
        (dict(top_k=0), INVALID, "top_k"), (dict(top_k=(1 << 20) + 1), UNSUPPORTED, "top_k"), (dict(selected=None), INVALID, "selected"),
        (dict(o=None), INVALID, "o is NULL"), (dict(ws=None), WORKSPACE, "workspace"), (dict(ws_bytes=need - 1), WORKSPACE, "workspace"),
        (dict(lse=base["o"]), INVALID, "aliases"), (dict(batch=0, q=None), OK, ""),
    ] + _aliases(base, ["o", "lse", "ws"], {"q": "q", "k": "k_cache", "v": "v_cache", "table": "block_table", "lens": "lens",
                                            "selected": "selected"}))


MASS = ["q", "k", "lse", "mass", "table", "starts", "positions", "len_old", "lens", "tokens", "batch", "H", "n_kv", "d", "max_pages",
        "table_stride"] + CACHE + ["q_sr", "q_sh"] + STRIDES + ["scale", "k_scale", "dtype", "kv", "stream"]


def test_mass_checks(lib):
    base = _base(MASS, 9, tokens=5)
    _table(lib, "ssm_kv_mass_update", MASS, base, PAGED + STRIDED + HEADS + SCALES + [
        (dict(tokens=-1), INVALID, "must be >= 0"), (dict(tokens=1 << 28), UNSUPPORTED, "too large"), (dict(lse=None), INVALID, "lse is NULL"),
        (dict(mass=None), INVALID, "mass is NULL"), (dict(starts=None), INVALID, "starts"), (dict(positions=None), INVALID, "positions"),
        (dict(len_old=None), INVALID, "len_old"), (dict(mass=ctypes.c_void_p(0x200002)), UNSUPPORTED, "mass is not aligned"),
        (dict(batch=0, q=None, tokens=0), OK, ""),
    ] + _aliases(base, ["mass"], {"q": "q", "k": "k_cache", "lse": "lse", "table": "block_table", "starts": "starts",
                                  "positions": "positions", "len_old": "len_old", "lens": "lens"}))


EVICT = ["k", "v", "mass", "table", "lens", "len_out", "kept", "batch", "n_kv", "d", "max_pages", "table_stride"] + CACHE + [
         "budget", "recent"] + STRIDES + ["kv", "stream"]


def test_evict_checks(lib):
    base = _base(EVICT, 7, budget=10, recent=2)
    outs = {"k": "k_cache", "v": "v_cache", "mass": "mass", "len_out": "len_out", "kept": "kept"}
    _table(lib, "ssm_kv_evict", EVICT, base, PAGED + STRIDED + [
        (dict(kv=3), INVALID, "kv_dtype 3"), (dict(budget=0, recent=0), INVALID, "budget"), (dict(recent=-1), INVALID, "recent"),
        (dict(recent=11), INVALID, "recent 11 > budget 10"), (dict(budget=1 << 31), UNSUPPORTED, "too large"),
        (dict(kept=None), INVALID, "kept is NULL"), (dict(len_out=None), INVALID, "len_out is NULL"), (dict(v=None), INVALID, "v_cache"),
        (dict(v=ctypes.c_void_p(0x200008)), UNSUPPORTED, "v_cache is not 16"), (dict(mass=ctypes.c_void_p(0x200001)), UNSUPPORTED, "mass"),
        (dict(batch=0, k=None), OK, ""),
    ] + _aliases(base, outs, {"table": "block_table", "lens": "lens"})
        + [({b: base[a]}, INVALID, "aliases") for a in outs for b in outs if a != b])


def test_the_bindings_own_checks(m):
    f, b, i = torch.float32, torch.bfloat16, torch.int32
    z = lambda *s, t=f: torch.zeros(s, dtype=t)  # noqa: E731
    c = z(4, 16, 1, 8)
    common = [(dict(k_cache=z(4, 16, 1, 8, t=torch.float16)), TypeError, "k_cache: dtype"), (dict(k_cache=z(4, 16, 8)), ValueError, "k_cache: shape"),
              (dict(k_cache=None), TypeError, "k_cache: a tensor")]
    rows = [(dict(q=z(2, 2, 16)), ValueError, "headdim"), (dict(q=z(2, 16)), ValueError, "q: shape"),
            (dict(q=z(2, 2, 8, t=torch.float16)), TypeError, "q: dtype"), (dict(q=z(2, 8, 2).transpose(1, 2)), ValueError, "last dim")]

    def each(fn, base, cases):
        for kw, err, word in cases + [({}, ValueError, "expected a GPU")]:
            with pytest.raises(err, match=word):
                fn(**dict(base, **kw))

    lens, table = z(2, t=i), z(2, 5, t=i)
    attn = dict(q=z(2, 2, 8), k_cache=c, v_cache=c.clone(), block_table=table, lens=lens, scale=1.0)
    each(m.ssm_prefix_attn_decode_fwd, dict(attn, prefix=lens, prefix_table=z(3, 7, t=i), prefix_lens=z(3, t=i)), common + rows + [
        (dict(prefix=z(3, t=i)), ValueError, "prefix: shape"), (dict(prefix_lens=z(2, t=i)), ValueError, "prefix_lens: shape"),
        (dict(prefix_table=z(3, t=i)), ValueError, "prefix_table: shape"), (dict(block_table=z(3, 5, t=i)), ValueError, "block_table: 3 rows"),
        (dict(v_cache=z(4, 16, 3, 8)[:, :, 1:2]), ValueError, "strides"), (dict(scale="x"), TypeError, "scale: a number")])
    each(m.ssm_select_attn_decode_fwd, dict(attn, selected=z(2, 1, 4, t=i)), common + rows + [
        (dict(selected=z(2, 2, 4, t=i)), ValueError, "selected: shape"), (dict(selected=z(2, 1, 4, t=torch.int64)), TypeError, "selected: dtype"),
        (dict(selected=z(2, 4, t=i)), ValueError, "selected: shape"), (dict(lens=z(3, t=i)), ValueError, "lens: shape")])
    each(m.ssm_kv_page_bounds_update, dict(k_cache=c, bounds=z(4, 1, 2, 8), block_table=table, len_old=lens, lens=lens), common + [
        (dict(bounds=z(4, 1, 2, 8, t=b)), TypeError, "bounds: dtype"), (dict(bounds=z(4, 2, 1, 8)), ValueError, "bounds: shape"),
        (dict(len_old=z(3, t=i)), ValueError, "len_old: shape"), (dict(block_table=z(2, 5)), TypeError, "block_table: dtype")])
    each(m.ssm_kv_page_select_fwd, dict(q=z(2, 2, 8), bounds=z(4, 1, 2, 8), block_table=table, lens=lens, page_size=16, top_k=3), [
        (dict(bounds=z(4, 1, 2, 16)), ValueError, "bounds: shape"), (dict(bounds=z(4, 1, 2, 8, t=i)), TypeError, "bounds: dtype"),
        (dict(top_k=0), ValueError, "top_k"), (dict(top_k=1.5), TypeError, "top_k"), (dict(page_size="x"), TypeError, "page_size"),
        (dict(selected=z(2, 1, 4, t=i)), ValueError, "selected: shape")])
    each(m.ssm_kv_mass_update, dict(q=z(3, 2, 8), k_cache=c, lse=z(3, 2), mass=z(4, 1, 16), block_table=table, starts=z(3, t=i),
                                    positions=z(3, t=i), len_old=lens, lens=lens, scale=1.0), common + [
        (dict(lse=z(3, 1)), ValueError, "lse: shape"), (dict(mass=z(4, 16, 1)), ValueError, "mass: shape"),
        (dict(starts=z(2, t=i)), ValueError, "starts: shape"), (dict(positions=z(2, t=i)), ValueError, "positions: shape"),
        (dict(mass=z(4, 1, 32)[..., ::2]), ValueError, "mass must be contiguous")])
    each(m.ssm_kv_evict, dict(k_cache=c, v_cache=c.clone(), mass=z(4, 1, 16), block_table=table, lens=lens, budget=4), common + [
        (dict(budget=0), ValueError, "budget"), (dict(recent=None), TypeError, "recent"), (dict(mass=z(4, 1, 16, t=b)), TypeError, "mass: dtype"),
        (dict(kept=z(2, 1, 5, t=i)), ValueError, "kept: shape|expected a GPU")])
    for flag in (z(2),):
        with pytest.raises(RuntimeError, match="ambiguous"):
            m.ssm_select_attn_decode_fwd(**attn, selected=z(2, 1, 4, t=i), return_lse=flag)
