"""Long contexts in the paged key-value cache of the attention operators: rows that share a long
prefix, attention over the pages that a cheap score selects, and eviction of the tokens that
gathered the least attention weight.

Binding of include/ssm_longctx.h in the manner and the compiled module of attn.py.
"""
from __future__ import annotations

import ctypes

from . import _I, _Z, _lib
from .attn import _bind, _done

__all__ = [
    "ssm_prefix_attn_decode_fwd", "ssm_prefix_attn_decode_fwd_workspace_size", "ssm_kv_page_bounds_update",
    "ssm_kv_page_select_fwd", "ssm_kv_page_select_fwd_workspace_size", "ssm_select_attn_decode_fwd",
    "ssm_select_attn_decode_fwd_workspace_size", "ssm_kv_mass_update", "ssm_kv_evict",
]

_lib.ssm_prefix_attn_decode_fwd_workspace_size.argtypes = [_I] * 7
_lib.ssm_prefix_attn_decode_fwd_workspace_size.restype = _Z
_lib.ssm_kv_page_select_fwd_workspace_size.argtypes = [_I] * 4
_lib.ssm_kv_page_select_fwd_workspace_size.restype = _Z
_lib.ssm_select_attn_decode_fwd_workspace_size.argtypes = [_I] * 7
_lib.ssm_select_attn_decode_fwd_workspace_size.restype = _Z


def _finished(rc):
    _done(rc)


def ssm_prefix_attn_decode_fwd_workspace_size(batch, n_heads, n_kv_heads, headdim, max_prefix_pages, max_pages,
                                              page_size) -> int:
    return int(_lib.ssm_prefix_attn_decode_fwd_workspace_size(batch, n_heads, n_kv_heads, headdim, max_prefix_pages,
                                                              max_pages, page_size))


def ssm_prefix_attn_decode_fwd(q, k_cache, v_cache, prefix, prefix_table, prefix_lens, block_table, lens, *, scale,
                               k_scale=1.0, v_scale=1.0, return_lse=False, o=None, lse=None, workspace=None):
    """ssm_paged_attn_decode_fwd for rows that share prefixes: row r attends to the tokens of
    prefix[r] (batch,) int32 (outside 0..prefixes-1: none) and then to its own.  prefix_table
    (prefixes, max_prefix_pages) and prefix_lens (prefixes,) int32 hold the prefixes' pages and
    tokens; block_table (batch, max_pages) and lens (batch,) int32 the rows' own, counted from the
    prefix's end.  Rows of one prefix cost least next to each other.  Returns o (batch, H, d) in q's
    dtype, or (o, lse) with lse (batch, H) fp32.  `workspace`: a uint8 tensor of
    ssm_prefix_attn_decode_fwd_workspace_size bytes."""
    return _done(_bind.prefix_attn_fwd(q, k_cache, v_cache, prefix, prefix_table, prefix_lens, block_table, lens, scale, k_scale,
                                       v_scale, return_lse, o, lse, workspace))


def ssm_kv_page_bounds_update(k_cache, bounds, block_table, len_old, lens) -> None:
    """Smallest and largest keys of the pages that the tokens len_old[r]..lens[r]-1 (batch,)
    int32 of each request stand on, into bounds (pages, Hk, 2, d) of k_cache's dtype, in place: of
    these tokens, and of what bounds held for a page that had tokens before."""
    _finished(_bind.page_bounds(k_cache, bounds, block_table, len_old, lens))


def ssm_kv_page_select_fwd_workspace_size(batch, n_kv_heads, max_pages, top_k) -> int:
    return int(_lib.ssm_kv_page_select_fwd_workspace_size(batch, n_kv_heads, max_pages, top_k))


def ssm_kv_page_select_fwd(q, bounds, block_table, lens, *, page_size, top_k, first=0, last=1, selected=None,
                           workspace=None):
    """The pages that each (row, kv head) is to look at: the `first` first and `last` last ones and
    those whose keys can have the largest products with the row's queries, top_k in all.  q (batch, H,
    d) fp32|bf16, strided; bounds as ssm_kv_page_bounds_update keeps them; block_table, lens as in
    ssm_paged_attn_decode_fwd.  Returns selected (batch, Hk, top_k) int32: places in the row's
    block table in rising order, -1 behind the last.  `workspace`: a uint8 tensor of
    ssm_kv_page_select_fwd_workspace_size bytes."""
    return _done(_bind.page_select(q, bounds, block_table, lens, page_size, top_k, first, last, selected, workspace))


def ssm_select_attn_decode_fwd_workspace_size(batch, n_heads, n_kv_heads, headdim, max_pages, page_size, top_k) -> int:
    return int(_lib.ssm_select_attn_decode_fwd_workspace_size(batch, n_heads, n_kv_heads, headdim, max_pages, page_size,
                                                              top_k))


def ssm_select_attn_decode_fwd(q, k_cache, v_cache, block_table, lens, selected, *, scale, k_scale=1.0, v_scale=1.0,
                               return_lse=False, o=None, lse=None, workspace=None):
    """ssm_paged_attn_decode_fwd over the tokens of chosen pages alone: selected (batch, Hk,
    top_k) int32 as ssm_kv_page_select_fwd gives it.  `workspace`: a uint8 tensor of
    ssm_select_attn_decode_fwd_workspace_size bytes."""
    return _done(_bind.select_attn_fwd(q, k_cache, v_cache, block_table, lens, selected, scale, k_scale, v_scale, return_lse, o,
                                       lse, workspace))


def ssm_kv_mass_update(q, k_cache, lse, mass, block_table, starts, positions, len_old, lens, *, scale, k_scale=1.0) -> None:
    """Adds the softmax weights of a step's queries to each cached token's running sum, mass
    (pages, Hk, page_size) fp32, in place.  q (tokens, H, d) and lse (tokens, H) fp32 of the step's
    rows; request r has rows starts[r]..starts[r+1]-1, row t at place positions[t] of its cache
    (what ssm_kv_pages_step returns); tokens from len_old[r] to lens[r] - 1 are new and start from 0.
    lse is that of attention over all the tokens that a row sees, not over chosen pages or a window."""
    _finished(_bind.mass_update(q, k_cache, lse, mass, block_table, starts, positions, len_old, lens, scale, k_scale))


def ssm_kv_evict(k_cache, v_cache, mass, block_table, lens, *, budget, recent=0, len_out=None, kept=None):
    """Cuts each request of more than `budget` tokens to that many, for each kv head the last
    `recent` tokens and those of the largest mass, moved forward in their order (k_cache, v_cache and
    mass in place).  Returns (len_out (batch,), kept (batch, Hk, budget)) int32: the tokens that
    requests have now, and the place that each had before (-1 behind the last).  Pass lens and
    len_out to ssm_kv_pages_step as len_old and len_new to free the pages."""
    return _done(_bind.evict(k_cache, v_cache, mass, block_table, lens, budget, recent, len_out, kept))
