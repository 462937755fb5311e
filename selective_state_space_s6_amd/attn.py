"""Paged attention for the attention layers between state-space layers: the cache's pages,
norm and rotation of the heads that enter it, and attention of one new token over it.

Binding of include/ssm_attn.h in the package's manner (the names of the C entry points,
dtype and shape checks here, everything else in the library, the current HIP stream); it
differs in that q, k, v and the caches may be strided views.
"""
from __future__ import annotations

import ctypes

import torch

from . import _I, _P, _Z, _check, _lib

__all__ = [
    "ssm_kv_pages_step", "ssm_qk_norm_rope_fwd", "ssm_qk_norm_rope_bwd", "ssm_qk_norm_rope_bwd_workspace_size",
    "ssm_qk_norm_rope_cache_fwd", "ssm_paged_attn_decode_fwd", "ssm_paged_attn_decode_fwd_workspace_size",
    "SSM_ROPE_INTERLEAVED", "SSM_QK_NO_NORM", "SSM_KV_F32", "SSM_KV_BF16", "SSM_KV_F8E4M3",
]

SSM_ROPE_INTERLEAVED, SSM_QK_NO_NORM = 0x1, 0x2
SSM_KV_F32, SSM_KV_BF16, SSM_KV_F8E4M3 = 0, 1, 2

_F, _D, _U = ctypes.c_float, ctypes.c_int, ctypes.c_uint32
_lib.ssm_kv_pages_step.argtypes = [_P] * 12 + [_I] * 6 + [_P]
_lib.ssm_qk_norm_rope_fwd.argtypes = [_P] * 8 + [_I] * 9 + [_F, _D, _U, _P]
_lib.ssm_qk_norm_rope_bwd.argtypes = [_P] * 12 + [_I] * 13 + [_F, _D, _U, _P, _Z, _P]
_lib.ssm_qk_norm_rope_bwd_workspace_size.argtypes = [_I] * 4 + [_U]
_lib.ssm_qk_norm_rope_bwd_workspace_size.restype = _Z
_lib.ssm_qk_norm_rope_cache_fwd.argtypes = [_P] * 11 + [_I] * 16 + [_F] * 3 + [_D, _D, _U, _P]
_lib.ssm_paged_attn_decode_fwd.argtypes = [_P] * 7 + [_I] * 13 + [_F, _I, _F, _F, _D, _D, _P, _Z, _P]
_lib.ssm_paged_attn_decode_fwd_workspace_size.argtypes = [_I] * 6
_lib.ssm_paged_attn_decode_fwd_workspace_size.restype = _Z
for _n in ("ssm_kv_pages_step", "ssm_qk_norm_rope_fwd", "ssm_qk_norm_rope_bwd", "ssm_qk_norm_rope_cache_fwd",
           "ssm_paged_attn_decode_fwd"):
    getattr(_lib, _n).restype = ctypes.c_int

_i32, _i64, _f32, _bf16 = torch.int32, torch.int64, torch.float32, torch.bfloat16
_DTYPE = {_f32: 0, _bf16: 1}
_KV_DTYPE = {_f32: SSM_KV_F32, _bf16: SSM_KV_BF16, torch.float8_e4m3fn: SSM_KV_F8E4M3}


def _want(t, name, dtype, shape, dev):
    """The address of a contiguous tensor of this dtype, shape and device."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _view(t, name, dtype, shape, dev):
    """The address and strides of a tensor whose last dim has stride 1."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    s = t.stride()
    if s[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name}: the last dim must have stride 1")
    return t.data_ptr(), s


def _dtype(t, name):
    d = _DTYPE.get(t.dtype)
    if d is None:
        raise TypeError(f"{name}: dtype {t.dtype}, expected float32 or bfloat16")
    return d


def _gpu(dev):
    if dev.type != "cuda":
        raise ValueError(f"tensors are on {dev}, expected a GPU")
    return torch.cuda.current_stream(dev).cuda_stream


def ssm_kv_pages_step(len_old, len_new, block_table, free_ring, ring, *, page_size, n_tokens):
    """One scheduling step of a paged cache.  len_old, len_new (batch,) int32: tokens each
    request has and is to have; block_table (batch, max_pages) int32 and free_ring (n_pages,)
    int32, both updated in place; ring (2,) int32 = [head, free].  n_tokens: room for the new
    tokens' maps.  Returns a dict: ring (2,), len (batch,) now held, starts (batch + 1,),
    request, positions (n_tokens,) int32, slots (n_tokens,) int64 (-1 past the last new token,
    and slots of requests that got no pages), denied (1,) refused requests.  Nothing is copied
    to the host; pass `len` and `ring` to the next step."""
    dev = len_old.device
    batch, max_pages = block_table.shape
    n_pages = free_ring.shape[0]
    shape = (batch,)
    p_old, p_new = _want(len_old, "len_old", _i32, shape, dev), _want(len_new, "len_new", _i32, shape, dev)
    p_table, st = _view(block_table, "block_table", _i32, (batch, max_pages), dev)
    p_free = _want(free_ring, "free_ring", _i32, (n_pages,), dev)
    p_ring = _want(ring, "ring", _i32, (2,), dev)
    stream = _gpu(dev)
    n_tokens = int(n_tokens)
    new = lambda n, dtype=_i32: torch.empty(n, dtype=dtype, device=dev)  # noqa: E731
    ring_out, length, starts, denied = new(2), new(batch), new(batch + 1), new(1)
    request, positions, slots = new(max(n_tokens, 0)), new(max(n_tokens, 0)), new(max(n_tokens, 0), _i64)
    _check(_lib.ssm_kv_pages_step(p_old, p_new, p_table, p_free, p_ring, ring_out.data_ptr(), length.data_ptr(),
                                  starts.data_ptr(), request.data_ptr(), positions.data_ptr(), slots.data_ptr(),
                                  denied.data_ptr(), batch, max_pages, st[0] if batch > 1 else max_pages, n_pages,
                                  page_size, n_tokens, stream))
    return {"ring": ring_out, "len": length, "starts": starts, "request": request, "positions": positions,
            "slots": slots, "denied": denied}


def _rope_args(q, k, wq, wk, inv_freq, positions, flags):
    """Checked addresses, strides and sizes that the norm and rotation calls share."""
    dev, dty = q.device, q.dtype
    T, H, d = q.shape
    dt = _dtype(q, "q")
    pq, sq = _view(q, "q", dty, (T, H, d), dev)
    pk, sk, Hk = None, (0, 0, 1), 0
    if k is not None:
        Hk = k.shape[1]
        pk, sk = _view(k, "k", dty, (T, Hk, d), dev)
    pwq = pwk = None
    if not flags & SSM_QK_NO_NORM:
        pwq = _want(wq, "wq", _f32, (d,), dev)
        pwk = _want(wk, "wk", _f32, (d,), dev) if k is not None else None
    half = inv_freq.shape[0]
    pf, pp = _want(inv_freq, "inv_freq", _f32, (half,), dev), _want(positions, "positions", _i32, (T,), dev)
    return dev, dty, dt, T, H, Hk, d, 2 * half, pq, sq, pk, sk, pwq, pwk, pf, pp


def ssm_qk_norm_rope_fwd(q, k, wq, wk, inv_freq, positions, *, eps=1e-6, flags=0, q_out=None, k_out=None):
    """RMS norm of each q and k head and position rotation in one pass.  q (T, H, d), k
    (T, Hk, d) fp32|bf16, strided (k may be None); wq, wk (d,) fp32 (not read under
    SSM_QK_NO_NORM); inv_freq (rot/2,) fp32: the first rot values of a head turn by
    positions (T,) int32 times it.  Returns (q_out, k_out), contiguous; q_out=q and k_out=k
    work in place on contiguous tensors."""
    dev, dty, dt, T, H, Hk, d, rot, pq, sq, pk, sk, pwq, pwk, pf, pp = _rope_args(q, k, wq, wk, inv_freq, positions, flags)
    if q_out is None:
        q_out = torch.empty((T, H, d), dtype=dty, device=dev)
    poq, pok = _want(q_out, "q_out", dty, (T, H, d), dev), None
    if k is not None:
        if k_out is None:
            k_out = torch.empty((T, Hk, d), dtype=dty, device=dev)
        pok = _want(k_out, "k_out", dty, (T, Hk, d), dev)
    _check(_lib.ssm_qk_norm_rope_fwd(pq, pk, pwq, pwk, pf, pp, poq, pok, T, H, Hk, d, rot, sq[0], sq[1], sk[0], sk[1],
                                     eps, dt, flags, _gpu(dev)))
    return q_out, k_out


def ssm_qk_norm_rope_bwd_workspace_size(n_tokens, n_heads, n_kv_heads, headdim, flags=0) -> int:
    return int(_lib.ssm_qk_norm_rope_bwd_workspace_size(n_tokens, n_heads, n_kv_heads, headdim, flags))


def ssm_qk_norm_rope_bwd(q, k, wq, wk, inv_freq, positions, dq_out, dk_out, *, eps=1e-6, flags=0, out=None,
                         workspace=None):
    """Gradients of ssm_qk_norm_rope_fwd.  Inputs as there, plus the cotangents dq_out, dk_out
    in q's and k's shapes and dtype, strided.  Returns a dict: dq, dk in q's dtype; dwq, dwk
    (d,) fp32 (None under SSM_QK_NO_NORM, as the k ones are without k).  `out` may hold
    preallocated tensors under those names (dq may be dq_out, dk may be dk_out); `workspace`
    a uint8 tensor of ssm_qk_norm_rope_bwd_workspace_size bytes."""
    dev, dty, dt, T, H, Hk, d, rot, pq, sq, pk, sk, pwq, pwk, pf, pp = _rope_args(q, k, wq, wk, inv_freq, positions, flags)
    pgq, gq = _view(dq_out, "dq_out", dty, (T, H, d), dev)
    pgk, gk = _view(dk_out, "dk_out", dty, (T, Hk, d), dev) if k is not None else (None, (0, 0, 1))
    norm = not flags & SSM_QK_NO_NORM
    g = dict(out or {})
    at = {}
    for n, shape, dtype, used in (("dq", (T, H, d), dty, True), ("dk", (T, Hk, d), dty, k is not None),
                                  ("dwq", (d,), _f32, norm), ("dwk", (d,), _f32, norm and k is not None)):
        if not used:
            g[n] = at[n] = None
            continue
        if g.get(n) is None:
            g[n] = torch.empty(shape, dtype=dtype, device=dev)
        at[n] = _want(g[n], n, dtype, shape, dev)
    need = int(_lib.ssm_qk_norm_rope_bwd_workspace_size(T, H, Hk, d, flags))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    _check(_lib.ssm_qk_norm_rope_bwd(pq, pk, pwq, pwk, pf, pp, pgq, pgk, at["dq"], at["dk"], at["dwq"], at["dwk"],
                                     T, H, Hk, d, rot, sq[0], sq[1], sk[0], sk[1], gq[0], gq[1], gk[0], gk[1],
                                     eps, dt, flags, workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(), _gpu(dev)))
    return g


def _caches(k_cache, v_cache, dev):
    """Addresses, strides, sizes and type of a pair of caches (pages, page_size, Hk, d)."""
    shape, kv = k_cache.shape, _KV_DTYPE.get(k_cache.dtype)
    if kv is None:
        raise TypeError(f"k_cache: dtype {k_cache.dtype}, expected float32, bfloat16 or float8_e4m3fn")
    if len(shape) != 4:
        raise ValueError(f"k_cache: shape {tuple(shape)}, expected (pages, page_size, kv_heads, headdim)")
    pk, sk = _view(k_cache, "k_cache", k_cache.dtype, shape, dev)
    pv, sv = _view(v_cache, "v_cache", k_cache.dtype, shape, dev)
    if sk != sv:
        raise ValueError(f"v_cache: strides {sv}, expected k_cache's {sk}")
    return pk, pv, sk, shape, kv


def ssm_qk_norm_rope_cache_fwd(q, k, v, wq, wk, inv_freq, positions, slots, k_cache, v_cache, *, eps=1e-6,
                               k_scale=1.0, v_scale=1.0, flags=0, q_out=None):
    """ssm_qk_norm_rope_fwd for tokens that enter a paged cache: returns q_out, and writes the
    rotated k and the unchanged v (T, Hk, d) of token t at slots[t] (int64, page * page_size +
    place; others write nothing) of k_cache, v_cache (pages, page_size, Hk, d), any strides
    with the last one 1, in q's dtype or float8_e4m3fn (then stored as value / scale)."""
    dev, dty, dt, T, H, Hk, d, rot, pq, sq, pk, sk, pwq, pwk, pf, pp = _rope_args(q, k, wq, wk, inv_freq, positions, flags)
    pv, sv = _view(v, "v", dty, (T, Hk, d), dev)
    ps = _want(slots, "slots", _i64, (T,), dev)
    ck, cv, cs, shape, kv = _caches(k_cache, v_cache, dev)
    if shape[2] != Hk or shape[3] != d:
        raise ValueError(f"k_cache: shape {tuple(shape)}, expected (pages, page_size, {Hk}, {d})")
    if q_out is None:
        q_out = torch.empty((T, H, d), dtype=dty, device=dev)
    poq = _want(q_out, "q_out", dty, (T, H, d), dev)
    _check(_lib.ssm_qk_norm_rope_cache_fwd(pq, pk, pv, pwq, pwk, pf, pp, ps, poq, ck, cv, T, H, Hk, d, rot,
                                           shape[0], shape[1], sq[0], sq[1], sk[0], sk[1], sv[0], sv[1],
                                           cs[0], cs[1], cs[2], eps, k_scale, v_scale, dt, kv, flags, _gpu(dev)))
    return q_out


def ssm_paged_attn_decode_fwd_workspace_size(batch, n_heads, n_kv_heads, headdim, max_pages, page_size) -> int:
    return int(_lib.ssm_paged_attn_decode_fwd_workspace_size(batch, n_heads, n_kv_heads, headdim, max_pages, page_size))


def ssm_paged_attn_decode_fwd(q, k_cache, v_cache, block_table, lens, *, scale, window=0, k_scale=1.0, v_scale=1.0,
                              return_lse=False, o=None, lse=None, workspace=None):
    """Attention of one new token a row over a paged cache.  q (batch, H, d) fp32|bf16,
    strided; k_cache, v_cache (pages, page_size, Hk, d) in q's dtype or float8_e4m3fn with
    bf16 q (value = stored * scale); block_table (batch, max_pages) int32; lens (batch,)
    int32 cached tokens of each row; window > 0: the last `window` of them.  Returns o
    (batch, H, d) in q's dtype, or (o, lse) with lse (batch, H) fp32.  A row without tokens
    has o = 0, lse = -inf.  `workspace`: a uint8 tensor of
    ssm_paged_attn_decode_fwd_workspace_size bytes."""
    dev, dty = q.device, q.dtype
    B, H, d = q.shape
    dt = _dtype(q, "q")
    pq, sq = _view(q, "q", dty, (B, H, d), dev)
    ck, cv, cs, shape, kv = _caches(k_cache, v_cache, dev)
    n_pages, page_size, Hk, dc = shape
    if dc != d:
        raise ValueError(f"k_cache: shape {tuple(shape)}, expected headdim {d}")
    max_pages = block_table.shape[1]
    pt, st = _view(block_table, "block_table", _i32, (B, max_pages), dev)
    pl = _want(lens, "lens", _i32, (B,), dev)
    if o is None:
        o = torch.empty((B, H, d), dtype=dty, device=dev)
    po = _want(o, "o", dty, (B, H, d), dev)
    if return_lse and lse is None:
        lse = torch.empty((B, H), dtype=_f32, device=dev)
    ple = None if lse is None else _want(lse, "lse", _f32, (B, H), dev)
    if workspace is None:
        need = _lib.ssm_paged_attn_decode_fwd_workspace_size(B, H, Hk, d, max_pages, page_size)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    _check(_lib.ssm_paged_attn_decode_fwd(pq, ck, cv, pt, pl, po, ple, B, H, Hk, d, max_pages,
                                          st[0] if B > 1 else max_pages, n_pages, page_size, sq[0], sq[1],
                                          cs[0], cs[1], cs[2], scale, window, k_scale, v_scale, dt, kv,
                                          workspace.data_ptr(), workspace.numel() * workspace.element_size(), _gpu(dev)))
    return (o, lse) if lse is not None else o
