"""include/ssm_attn.h without a GPU: every declared symbol is exported, workspace sizes, and
every argument check returns its code and message before any HIP call (the addresses are
never dereferenced on these paths); the binding's own checks of dtype, shape, stride and
device."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssm_attn.h")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3


@pytest.fixture(scope="module")
def m():
    import selective_state_space_s6_amd as m
    return m


@pytest.fixture(scope="module")
def lib(m):
    L = ctypes.CDLL(m.LIB_PATH)
    I, P, Z, F, D, U = (ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float, ctypes.c_int, ctypes.c_uint32)
    L.ssm_last_error.restype = ctypes.c_char_p
    L.ssm_kv_pages_step.argtypes = [P] * 12 + [I] * 6 + [P]
    L.ssm_qk_norm_rope_fwd.argtypes = [P] * 8 + [I] * 9 + [F, D, U, P]
    L.ssm_qk_norm_rope_bwd.argtypes = [P] * 12 + [I] * 13 + [F, D, U, P, Z, P]
    L.ssm_qk_norm_rope_bwd_workspace_size.argtypes = [I] * 4 + [U]
    L.ssm_qk_norm_rope_bwd_workspace_size.restype = Z
    L.ssm_qk_norm_rope_cache_fwd.argtypes = [P] * 11 + [I] * 16 + [F] * 3 + [D, D, U, P]
    L.ssm_paged_attn_decode_fwd.argtypes = [P] * 7 + [I] * 13 + [F, I, F, F, D, D, P, Z, P]
    L.ssm_paged_attn_decode_fwd_workspace_size.argtypes = [I] * 6
    L.ssm_paged_attn_decode_fwd_workspace_size.restype = Z
    return L


def _p(i):
    return ctypes.c_void_p(0x100000 * (i + 1))


def _err(lib):
    return lib.ssm_last_error().decode()


def test_every_declared_symbol_is_exported(m, lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(ssm_\w+)\s*\(", text))
    assert names == {"ssm_kv_pages_step", "ssm_qk_norm_rope_fwd", "ssm_qk_norm_rope_bwd",
                     "ssm_qk_norm_rope_bwd_workspace_size", "ssm_qk_norm_rope_cache_fwd",
                     "ssm_paged_attn_decode_fwd", "ssm_paged_attn_decode_fwd_workspace_size"}
    for n in names:
        assert hasattr(lib, n) and n in m.__all__ and callable(getattr(m, n))


def _call(lib, fn, order, base, **kw):
    a = dict(base, **kw)
    assert set(a) == set(order)
    return getattr(lib, fn)(*(a[n] for n in order))


def _table(lib, fn, order, base, cases):
    for kw, code, word in cases:
        assert _call(lib, fn, order, base, **kw) == code, (fn, kw, _err(lib))
        assert word in _err(lib) and _err(lib).startswith(fn), (kw, _err(lib))


PAGES = ["len_old", "len_new", "block_table", "free_ring", "ring", "ring_out", "len_out", "starts", "request", "positions",
         "slots", "denied", "batch", "max_pages", "table_stride", "n_pages", "page_size", "n_tokens", "stream"]


def test_pages_checks(lib):
    base = {n: _p(i) for i, n in enumerate(PAGES[:12])}
    base.update(batch=4, max_pages=8, table_stride=8, n_pages=32, page_size=16, n_tokens=4, stream=None)
    _table(lib, "ssm_kv_pages_step", PAGES, base, [
        (dict(len_old=None), INVALID, "len_old is NULL"), (dict(denied=None), INVALID, "denied is NULL"),
        (dict(slots=None), INVALID, "slots is NULL"), (dict(batch=0), INVALID, "batch"), (dict(page_size=0), INVALID, "page_size"),
        (dict(n_pages=-1), INVALID, "n_pages"), (dict(n_tokens=-1), INVALID, "n_tokens"),
        (dict(batch=4097), UNSUPPORTED, "batch"), (dict(table_stride=7), INVALID, "table_stride"),
        (dict(max_pages=1 << 30, table_stride=1 << 30), UNSUPPORTED, "too large"),
        (dict(n_pages=1 << 27), UNSUPPORTED, "too large"), (dict(n_tokens=1 << 31), UNSUPPORTED, "too large"),
        (dict(request=ctypes.c_void_p(0x100004)), UNSUPPORTED, "request is not 16-byte aligned"),
        (dict(ring_out=base["ring"]), INVALID, "ring_out aliases ring"),
        (dict(len_out=base["len_old"]), INVALID, "len_out aliases len_old"),
        (dict(free_ring=base["block_table"]), INVALID, "aliases"),
    ])


ROPE = ["q", "k", "wq", "wk", "inv_freq", "positions", "q_out", "k_out", "n_tokens", "n_heads", "n_kv_heads", "headdim",
        "rot_dim", "q_st", "q_sh", "k_st", "k_sh", "eps", "dtype", "flags", "stream"]
ROPE_CASES = [
    (dict(q=None), INVALID, "q is NULL"), (dict(k=None), INVALID, "k is NULL"), (dict(wq=None), INVALID, "wq is NULL"),
    (dict(wk=None), INVALID, "wk is NULL"), (dict(inv_freq=None), INVALID, "inv_freq is NULL"),
    (dict(positions=None), INVALID, "positions is NULL"), (dict(n_tokens=-1), INVALID, "n_tokens"),
    (dict(n_heads=0), INVALID, "n_heads"), (dict(headdim=0), INVALID, "headdim"), (dict(headdim=257), UNSUPPORTED, "headdim"),
    (dict(rot_dim=63), INVALID, "rot_dim"), (dict(rot_dim=66), INVALID, "rot_dim"), (dict(rot_dim=-2), INVALID, "rot_dim"),
    (dict(dtype=2), INVALID, "dtype"), (dict(flags=4), INVALID, "flags"), (dict(eps=-1.0), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"), (dict(n_tokens=1 << 40), UNSUPPORTED, "too large"),
    (dict(q=ctypes.c_void_p(0x100001)), UNSUPPORTED, "q is not aligned"),
]


def test_rope_checks(lib):
    base = {n: _p(i) for i, n in enumerate(ROPE[:8])}
    base.update(n_tokens=4, n_heads=2, n_kv_heads=1, headdim=64, rot_dim=64, q_st=256, q_sh=64, k_st=256, k_sh=64,
                eps=1e-6, dtype=1, flags=0, stream=None)
    _table(lib, "ssm_qk_norm_rope_fwd", ROPE, base, ROPE_CASES + [
        (dict(q_out=None), INVALID, "q_out is NULL"), (dict(k_out=None), INVALID, "k_out is NULL"),
        (dict(q_out=base["q"]), INVALID, "not contiguous"), (dict(k_out=base["k"]), INVALID, "not contiguous"),
        (dict(q_out=base["k"]), INVALID, "alias"), (dict(k_out=base["q_out"]), INVALID, "alias"),
    ])
    assert _call(lib, "ssm_qk_norm_rope_fwd", ROPE, base, n_tokens=0, q=None, k=None) == OK


BWD = ["q", "k", "wq", "wk", "inv_freq", "positions", "dq_out", "dk_out", "dq", "dk", "dwq", "dwk", "n_tokens", "n_heads",
       "n_kv_heads", "headdim", "rot_dim", "q_st", "q_sh", "k_st", "k_sh", "dq_st", "dq_sh", "dk_st", "dk_sh", "eps", "dtype",
       "flags", "workspace", "workspace_bytes", "stream"]


def test_rope_bwd_checks(lib):
    need = lib.ssm_qk_norm_rope_bwd_workspace_size(4, 2, 1, 64, 0)
    assert need > 0 and need % (64 * 4) == 0
    assert lib.ssm_qk_norm_rope_bwd_workspace_size(4, 2, 1, 64, 2) == 0          # no norm, no dw
    assert lib.ssm_qk_norm_rope_bwd_workspace_size(0, 2, 1, 64, 0) == 0
    # bounded by the chip, not by the tokens
    assert lib.ssm_qk_norm_rope_bwd_workspace_size(1 << 20, 16, 4, 128, 0) <= 1024 * 128 * 4
    base = {n: _p(i) for i, n in enumerate(BWD[:12])}
    base.update(n_tokens=4, n_heads=2, n_kv_heads=1, headdim=64, rot_dim=64, q_st=256, q_sh=64, k_st=256, k_sh=64,
                dq_st=256, dq_sh=64, dk_st=256, dk_sh=64, eps=1e-6, dtype=1, flags=0, workspace=_p(20), workspace_bytes=need,
                stream=None)
    _table(lib, "ssm_qk_norm_rope_bwd", BWD, base, ROPE_CASES + [
        (dict(dq_out=None), INVALID, "dq_out is NULL"), (dict(dk=None), INVALID, "dk is NULL"),
        (dict(dwq=None), INVALID, "dwq is NULL"), (dict(dq=base["dq_out"]), INVALID, "not contiguous"),
        (dict(dq=base["q"]), INVALID, "dq aliases q"), (dict(dwk=base["dwq"]), INVALID, "alias"),
        (dict(workspace=None), WORKSPACE, "workspace"), (dict(workspace_bytes=need - 1), WORKSPACE, "workspace"),
        (dict(workspace=ctypes.c_void_p(0x100004)), UNSUPPORTED, "workspace is not 16-byte aligned"),
    ])


CACHE = ["q", "k", "v", "wq", "wk", "inv_freq", "positions", "slots", "q_out", "k_cache", "v_cache", "n_tokens", "n_heads",
         "n_kv_heads", "headdim", "rot_dim", "n_pages", "page_size", "q_st", "q_sh", "k_st", "k_sh", "v_st", "v_sh", "c_sp",
         "c_st", "c_sh", "eps", "k_scale", "v_scale", "dtype", "kv_dtype", "flags", "stream"]


def test_cache_checks(lib):
    base = {n: _p(i) for i, n in enumerate(CACHE[:11])}
    base.update(n_tokens=4, n_heads=2, n_kv_heads=1, headdim=64, rot_dim=64, n_pages=8, page_size=16, q_st=256, q_sh=64,
                k_st=256, k_sh=64, v_st=256, v_sh=64, c_sp=1024, c_st=64, c_sh=64, eps=1e-6, k_scale=1.0, v_scale=1.0, dtype=1,
                kv_dtype=2, flags=0, stream=None)
    _table(lib, "ssm_qk_norm_rope_cache_fwd", CACHE, base, [c for c in ROPE_CASES if c[0] != dict(dtype=2)] + [
        (dict(v=None), INVALID, "v is NULL"), (dict(slots=None), INVALID, "slots is NULL"),
        (dict(k_cache=None), INVALID, "k_cache is NULL"), (dict(n_kv_heads=0), INVALID, "n_kv_heads"),
        (dict(kv_dtype=0), UNSUPPORTED, "kv_dtype"), (dict(dtype=0), UNSUPPORTED, "kv_dtype"),
        (dict(k_scale=0.0), INVALID, "scale"), (dict(v_scale=float("inf")), INVALID, "scale"),
        (dict(n_pages=0), INVALID, "n_pages"), (dict(page_size=1 << 29), UNSUPPORTED, "2^31"),
        (dict(c_sp=-1), INVALID, "strides"), (dict(c_sp=1 << 40), UNSUPPORTED, "extent"),
        (dict(v_cache=base["k_cache"]), INVALID, "alias"), (dict(k_cache=base["v"]), INVALID, "alias"),
        (dict(q_out=base["q"]), INVALID, "not contiguous"),
    ])


ATTN = ["q", "k_cache", "v_cache", "block_table", "lens", "o", "lse", "batch", "n_heads", "n_kv_heads", "headdim", "max_pages",
        "table_stride", "n_pages", "page_size", "q_sr", "q_sh", "c_sp", "c_st", "c_sh", "scale", "window", "k_scale", "v_scale",
        "dtype", "kv_dtype", "workspace", "workspace_bytes", "stream"]


def test_attn_checks(lib):
    need = lib.ssm_paged_attn_decode_fwd_workspace_size(4, 8, 2, 64, 8, 16)
    assert need > 0
    assert lib.ssm_paged_attn_decode_fwd_workspace_size(4, 8, 3, 64, 8, 16) == 0
    assert lib.ssm_paged_attn_decode_fwd_workspace_size(0, 8, 2, 64, 8, 16) == 0
    # bounded by the chip, not by the cache
    assert lib.ssm_paged_attn_decode_fwd_workspace_size(256, 64, 8, 128, 1 << 16, 16) < 24 << 20
    base = {n: _p(i) for i, n in enumerate(ATTN[:7])}
    base.update(batch=4, n_heads=8, n_kv_heads=2, headdim=64, max_pages=8, table_stride=8, n_pages=32, page_size=16, q_sr=512,
                q_sh=64, c_sp=2048, c_st=128, c_sh=64, scale=0.125, window=0, k_scale=1.0, v_scale=1.0, dtype=1, kv_dtype=1,
                workspace=_p(20), workspace_bytes=need, stream=None)
    mis = ctypes.c_void_p(0x100008)
    _table(lib, "ssm_paged_attn_decode_fwd", ATTN, base, [
        (dict(q=None), INVALID, "q is NULL"), (dict(k_cache=None), INVALID, "k_cache is NULL"),
        (dict(block_table=None), INVALID, "block_table is NULL"), (dict(lens=None), INVALID, "lens is NULL"),
        (dict(o=None), INVALID, "o is NULL"), (dict(batch=-1), INVALID, "batch"), (dict(n_heads=0), INVALID, "n_heads"),
        (dict(n_kv_heads=3), INVALID, "multiple"), (dict(headdim=264), UNSUPPORTED, "headdim"),
        (dict(headdim=60), UNSUPPORTED, "headdim"), (dict(headdim=72, kv_dtype=2), UNSUPPORTED, "headdim"),
        (dict(max_pages=0), INVALID, "max_pages"), (dict(table_stride=7), INVALID, "table_stride"),
        (dict(window=-1), INVALID, "window"), (dict(scale=float("nan")), INVALID, "scale"),
        (dict(kv_dtype=2, k_scale=-1.0), INVALID, "scale"), (dict(dtype=3), INVALID, "dtype"),
        (dict(dtype=0), UNSUPPORTED, "kv_dtype"), (dict(kv_dtype=0), UNSUPPORTED, "kv_dtype"),
        (dict(n_pages=0), INVALID, "n_pages"), (dict(c_st=-8), INVALID, "strides"), (dict(c_sp=1 << 40), UNSUPPORTED, "extent"),
        (dict(max_pages=1 << 27, table_stride=1 << 27), UNSUPPORTED, "too large"),
        (dict(c_st=132), UNSUPPORTED, "stride of the caches"), (dict(q_sh=68), UNSUPPORTED, "stride of q"),
        (dict(q=mis), UNSUPPORTED, "q is not 16-byte aligned"), (dict(v_cache=mis), UNSUPPORTED, "v_cache is not"),
        (dict(o=base["q"]), INVALID, "o aliases q"), (dict(lse=base["o"]), INVALID, "alias"),
        (dict(workspace=None), WORKSPACE, "workspace"), (dict(workspace_bytes=need - 1), WORKSPACE, "workspace"),
    ])
    assert _call(lib, "ssm_paged_attn_decode_fwd", ATTN, base, batch=0, q=None) == OK


def test_the_bindings_own_checks(m):
    f, b, i = torch.float32, torch.bfloat16, torch.int32
    z = lambda *s, t=f: torch.zeros(s, dtype=t)  # noqa: E731
    rope = dict(q=z(3, 2, 8), k=z(3, 1, 8), wq=z(8), wk=z(8), inv_freq=z(4), positions=z(3, t=i))
    for kw, err, word in [(dict(q=z(3, 2, 8, t=torch.float16)), TypeError, "q: dtype"), (dict(k=z(3, 1, 8, t=b)), TypeError, "k: dtype"),
                          (dict(k=z(2, 1, 8)), ValueError, "k: shape"), (dict(wq=z(7)), ValueError, "wq: shape"),
                          (dict(wk=z(8, t=b)), TypeError, "wk: dtype"), (dict(positions=z(3, t=torch.int64)), TypeError, "positions"),
                          (dict(q=z(3, 8, 2).transpose(1, 2)), ValueError, "last dim"), (dict(), ValueError, "expected a GPU")]:
        with pytest.raises(err, match=word):
            m.ssm_qk_norm_rope_fwd(**dict(rope, **kw))
    for flags in (1 << 32, -1):
        with pytest.raises(ValueError, match="flags"):
            m.ssm_qk_norm_rope_fwd(**rope, flags=flags)
    with pytest.raises(ValueError, match="dq_out: shape"):
        m.ssm_qk_norm_rope_bwd(**rope, dq_out=z(3, 1, 8), dk_out=z(3, 1, 8))
    c = z(4, 16, 1, 8)
    cache = dict(rope, v=z(3, 1, 8), slots=z(3, t=torch.int64), k_cache=c, v_cache=c.clone())
    for kw, err, word in [(dict(v=z(3, 2, 8)), ValueError, "v: shape"), (dict(slots=z(3, t=i)), TypeError, "slots"),
                          (dict(k_cache=z(4, 16, 2, 8), v_cache=z(4, 16, 2, 8)), ValueError, "k_cache: shape"),
                          (dict(v_cache=z(4, 1, 16, 8).permute(0, 2, 1, 3), k_cache=z(4, 16, 1, 16)[..., ::2]), ValueError, "last dim"),
                          (dict(k_cache=z(4, 16, 1, 8, t=torch.float16)), TypeError, "k_cache: dtype")]:
        with pytest.raises(err, match=word):
            m.ssm_qk_norm_rope_cache_fwd(**dict(cache, **kw))
    attn = dict(q=z(2, 2, 8), k_cache=c, v_cache=c.clone(), block_table=z(2, 5, t=i), lens=z(2, t=i), scale=1.0)
    for kw, err, word in [(dict(q=z(2, 2, 16)), ValueError, "headdim"), (dict(lens=z(3, t=i)), ValueError, "lens: shape"),
                          (dict(block_table=z(3, 5, t=i)), ValueError, "block_table: shape"),
                          (dict(v_cache=z(4, 16, 1, 8, t=b)), TypeError, "v_cache: dtype"),
                          (dict(v_cache=z(4, 16, 3, 8)[:, :, 1:2]), ValueError, "strides")]:
        with pytest.raises(err, match=word):
            m.ssm_paged_attn_decode_fwd(**dict(attn, **kw))
    with pytest.raises(ValueError, match="ring: shape"):
        m.ssm_kv_pages_step(z(2, t=i), z(2, t=i), z(2, 3, t=i), z(9, t=i), z(3, t=i), page_size=4, n_tokens=1)


def test_no_output_on_an_input_of_the_other_side(lib):
    """What one block writes while another still reads it is refused: an output or the workspace on any input but
    its own (dq on dq_out, dk on dk_out)."""
    need = lib.ssm_qk_norm_rope_bwd_workspace_size(4, 2, 2, 64, 0)
    base = {n: _p(i) for i, n in enumerate(BWD[:12])}
    base.update(n_tokens=4, n_heads=2, n_kv_heads=2, headdim=64, rot_dim=64, q_st=128, q_sh=64, k_st=128, k_sh=64,
                dq_st=128, dq_sh=64, dk_st=128, dk_sh=64, eps=1e-6, dtype=1, flags=0, workspace=_p(20), workspace_bytes=need,
                stream=None)
    own = {("dq", "dq_out"), ("dk", "dk_out")}
    ins = ["q", "k", "wq", "wk", "inv_freq", "positions", "dq_out", "dk_out"]
    _table(lib, "ssm_qk_norm_rope_bwd", BWD, base, [
        ({o: base[i]}, INVALID, f"{o} aliases {i}") for o in ("dq", "dk", "dwq", "dwk", "workspace") for i in ins if (o, i) not in own
    ] + [({"workspace": base[o]}, INVALID, "alias") for o in ("dq", "dk", "dwq", "dwk")])

    base = {n: _p(i) for i, n in enumerate(ROPE[:8])}
    base.update(n_tokens=4, n_heads=2, n_kv_heads=2, headdim=64, rot_dim=64, q_st=128, q_sh=64, k_st=128, k_sh=64,
                eps=1e-6, dtype=1, flags=0, stream=None)
    _table(lib, "ssm_qk_norm_rope_fwd", ROPE, base, [
        ({o: base[i]}, INVALID, f"{o} aliases {i}") for o in ("q_out", "k_out") for i in ("wq", "wk", "inv_freq", "positions")])

    base = {n: _p(i) for i, n in enumerate(CACHE[:11])}
    base.update(n_tokens=4, n_heads=2, n_kv_heads=1, headdim=64, rot_dim=64, n_pages=8, page_size=16, q_st=256, q_sh=64,
                k_st=256, k_sh=64, v_st=256, v_sh=64, c_sp=1024, c_st=64, c_sh=64, eps=1e-6, k_scale=1.0, v_scale=1.0, dtype=1,
                kv_dtype=2, flags=0, stream=None)
    _table(lib, "ssm_qk_norm_rope_cache_fwd", CACHE, base, [
        ({o: base[i]}, INVALID, f"{o} aliases {i}") for o in ("q_out", "k_cache", "v_cache") for i in ("inv_freq", "positions", "slots")])

    need = lib.ssm_paged_attn_decode_fwd_workspace_size(4, 8, 2, 64, 8, 16)
    base = {n: _p(i) for i, n in enumerate(ATTN[:7])}
    base.update(batch=4, n_heads=8, n_kv_heads=2, headdim=64, max_pages=8, table_stride=8, n_pages=32, page_size=16, q_sr=512,
                q_sh=64, c_sp=2048, c_st=128, c_sh=64, scale=0.125, window=0, k_scale=1.0, v_scale=1.0, dtype=1, kv_dtype=1,
                workspace=_p(20), workspace_bytes=need, stream=None)
    _table(lib, "ssm_paged_attn_decode_fwd", ATTN, base, [
        (dict(workspace=base[i]), INVALID, f"workspace aliases {i}") for i in ("q", "k_cache", "v_cache", "block_table", "lens")
    ] + [(dict(workspace=base[o]), INVALID, "alias") for o in ("o", "lse")])


def test_return_lse_that_is_no_truth_value(m):
    """A flag whose truth raises passes its own error on, not one about something else."""
    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t)  # noqa: E731
    with pytest.raises(RuntimeError, match="ambiguous"):
        m.ssm_paged_attn_decode_fwd(z(2, 2, 8), z(4, 16, 1, 8), z(4, 16, 1, 8), z(2, 5, t=torch.int32), z(2, t=torch.int32), scale=1.0,
                                    return_lse=z(2))
