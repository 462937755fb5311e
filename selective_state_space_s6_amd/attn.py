"""Paged attention for the attention layers between state-space layers: the cache's pages,
norm and rotation of the heads that enter it, and attention of one new token over it.

Binding of include/ssm_attn.h in the package's manner: the functions carry the names of
the C entry points, check dtypes, shapes and devices, allocate what the caller does not
pass, and hand addresses and the current HIP stream to the library.  It differs from the
scans' in two ways: q, k, v and the caches may be strided views, and the checks run in a
small compiled module (csrc/bind_attn.cpp), because these calls are short and frequent.
"""
from __future__ import annotations

import ctypes

from . import _I, _Z, _check, _lib

__all__ = [
    "ssm_kv_pages_step", "ssm_qk_norm_rope_fwd", "ssm_qk_norm_rope_bwd", "ssm_qk_norm_rope_bwd_workspace_size",
    "ssm_qk_norm_rope_cache_fwd", "ssm_paged_attn_decode_fwd", "ssm_paged_attn_decode_fwd_workspace_size",
    "SSM_ROPE_INTERLEAVED", "SSM_QK_NO_NORM", "SSM_KV_F32", "SSM_KV_BF16", "SSM_KV_F8E4M3",
]


class _NotLoaded:
    """In the compiled module's place where that is missing or was built for another torch: the scans,
    which do not need it, import all the same, and every call of this module raises."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"_attn_bind.so does not load ({self._why}): build it with `python "
                          "selective_state_space_s6_amd/build.py` (there is no non-HIP fallback)") from self._why


try:
    from . import _attn_bind as _bind
except ImportError as e:
    _bind = _NotLoaded(e)

SSM_ROPE_INTERLEAVED, SSM_QK_NO_NORM = 0x1, 0x2
SSM_KV_F32, SSM_KV_BF16, SSM_KV_F8E4M3 = 0, 1, 2

_lib.ssm_qk_norm_rope_bwd_workspace_size.argtypes = [_I] * 4 + [ctypes.c_uint32]
_lib.ssm_qk_norm_rope_bwd_workspace_size.restype = _Z
_lib.ssm_paged_attn_decode_fwd_workspace_size.argtypes = [_I] * 6
_lib.ssm_paged_attn_decode_fwd_workspace_size.restype = _Z


def _done(r):
    if type(r) is int:       # the library's status
        _check(r)
    return r


def ssm_kv_pages_step(len_old, len_new, block_table, free_ring, ring, *, page_size, n_tokens):
    """One scheduling step of a paged cache.  len_old, len_new (batch,) int32: tokens each
    request has and is to have; block_table (batch, max_pages) int32 and free_ring (n_pages,)
    int32, both updated in place; ring (2,) int32 = [head, free].  n_tokens: room for the new
    tokens' maps.  Returns a dict: ring (2,), len (batch,) now held, starts (batch + 1,),
    request, positions (n_tokens,) int32, slots (n_tokens,) int64 (-1 past the last new token,
    and slots of requests that got no pages), denied (1,) refused requests.  Nothing is copied
    to the host; pass `len` and `ring` to the next step."""
    return _done(_bind.pages_step(len_old, len_new, block_table, free_ring, ring, page_size, n_tokens))


def ssm_qk_norm_rope_fwd(q, k, wq, wk, inv_freq, positions, *, eps=1e-6, flags=0, q_out=None, k_out=None):
    """RMS norm of each q and k head and position rotation in one pass.  q (T, H, d), k
    (T, Hk, d) fp32|bf16, strided (k may be None); wq, wk (d,) fp32 (not read under
    SSM_QK_NO_NORM); inv_freq (rot/2,) fp32: the first rot values of a head turn by
    positions (T,) int32 times it.  Returns (q_out, k_out), contiguous; q_out=q and k_out=k
    work in place on contiguous tensors."""
    return _done(_bind.rope_fwd(q, k, wq, wk, inv_freq, positions, eps, flags, q_out, k_out))


def ssm_qk_norm_rope_bwd_workspace_size(n_tokens, n_heads, n_kv_heads, headdim, flags=0) -> int:
    return int(_lib.ssm_qk_norm_rope_bwd_workspace_size(n_tokens, n_heads, n_kv_heads, headdim, flags))


def ssm_qk_norm_rope_bwd(q, k, wq, wk, inv_freq, positions, dq_out, dk_out, *, eps=1e-6, flags=0, out=None,
                         workspace=None):
    """Gradients of ssm_qk_norm_rope_fwd.  Inputs as there, plus the cotangents dq_out, dk_out
    in q's and k's shapes and dtype, strided.  Returns a dict: dq, dk in q's dtype; dwq, dwk
    (d,) fp32 (None under SSM_QK_NO_NORM, as the k ones are without k).  `out` may hold
    preallocated tensors under those names (dq may be dq_out, dk may be dk_out); `workspace`
    a uint8 tensor of ssm_qk_norm_rope_bwd_workspace_size bytes."""
    g = out or {}
    return _done(_bind.rope_bwd(q, k, wq, wk, inv_freq, positions, dq_out, dk_out, eps, flags, g.get("dq"), g.get("dk"),
                                g.get("dwq"), g.get("dwk"), workspace))


def ssm_qk_norm_rope_cache_fwd(q, k, v, wq, wk, inv_freq, positions, slots, k_cache, v_cache, *, eps=1e-6,
                               k_scale=1.0, v_scale=1.0, flags=0, q_out=None):
    """ssm_qk_norm_rope_fwd for tokens that enter a paged cache: returns q_out, and writes the
    rotated k and the unchanged v (T, Hk, d) of token t at slots[t] (int64, page * page_size +
    place; others write nothing) of k_cache, v_cache (pages, page_size, Hk, d), any strides
    with the last one 1, in q's dtype or float8_e4m3fn (then stored as value / scale)."""
    return _done(_bind.rope_cache_fwd(q, k, wq, wk, inv_freq, positions, v, slots, k_cache, v_cache, eps, k_scale, v_scale,
                                      flags, q_out))


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
    return _done(_bind.attn_decode_fwd(q, k_cache, v_cache, block_table, lens, scale, window, k_scale, v_scale, return_lse,
                                       o, lse, workspace))
