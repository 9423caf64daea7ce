"""Serving over a paged KV cache: a step's plan, the norm and rotation of its
heads with the cache write, attention behind a shared prefix, drafted tokens,
and the keeping of pages.

The calls of ``include/rsa.h`` with the same names; as in the rest of the
binding they only check and marshal arguments, here in an extension module
(csrc/torch_paged.cpp), as a step makes many of them.  One decode step:

    plan = page_plan(cached_len, new_len, block_table, free_pages, page_size, n_pages, max_tokens, pos0=prefix_len)
    for each layer:
        q, _ = qk_norm_rope(q, k, wq, wk, plan.positions, cos_sin, v=v, slot_map=plan.slot_map,
                            k_cache=k_cache, v_cache=v_cache)
        out, lse = prefix_attn(q, k_cache, v_cache, plan.cu_new, block_table, plan.kv_len,
                               prefix_pages=prefix_pages, prefix_len=prefix_len)

With a tree of drafted tokens for every request (parent: each token's parent):

    plan = page_plan(...)
    tree = tree_plan(parent, plan.cu_new, plan.kv_len, max_tree, pos0=prefix_len)
    for each layer: qk_norm_rope as above with tree.positions, then
        out, lse = tree_attn(q, k_cache, v_cache, plan.cu_new, block_table, plan.kv_len, tree.mask, ...)
    new_len = cache_compact(k_caches, v_caches, block_table, cached_len, plan.kv_len, accepted, n_accepted)
    info = page_free(block_table, plan.kv_len, new_len, free_pages, plan.info[3:], page_size, n_pages)
    # the next step: cached_len = new_len, free_start = info[3:]

cache_compact also keeps a window of the cached tokens (cached_len 0, keep the window's tokens).  Keys keep
their rotation, and the plans go by lengths; from then on a request's new tokens are as many
positions further as it has dropped tokens (dropped int32 [R], on the device):

    row = torch.arange(max_tokens, device=dropped.device, dtype=torch.int32)
    request = torch.searchsorted(plan.cu_new[1:], row, right=True).clamp_(max=R - 1)
    positions = plan.positions + dropped[request]   # tree.positions in the same way

Caches are [n_pages, Hkv, page_size, d]; a step's rows are packed [T, H, d].
Nothing synchronises, so a step can be captured into a CUDA graph and replayed
with other lengths: what depends on them is read on the device.

No call takes part in autograd, as in the rest of the binding: inputs that
require a gradient are read like any others and results have no history.  A
training loop calls qk_norm_rope_bwd itself, for instance from the backward of
a torch.autograd.Function of its own.

Heads, NormRopeArgs and SIGS describe the C ABI for ctypes: load() types the
library's functions with them, for callers of the C calls themselves.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import threading
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import RSA_BF16, RSA_F32, RsaError, _build, load

PLAN_STATUS = {0: "ok", 1: "negative length", 2: "block table row too short", 3: "too few free pages",
               4: "more tokens than max_tokens", 5: "a fork's requests", 6: "no room for the free pages"}


class Heads(ctypes.Structure):
    """rsa_heads: a [T, H, d] operand with its token and head strides in elements."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class NormRopeArgs(ctypes.Structure):
    """rsa_qk_norm_rope_args."""
    _fields_ = [("dt", ctypes.c_int), ("T", ctypes.c_int64), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int),
                ("q", Heads), ("k", Heads), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int), ("n_axes", ctypes.c_int),
                ("sections", ctypes.c_int * 4), ("positions", ctypes.c_void_p), ("cos_sin", ctypes.c_void_p),
                ("max_pos", ctypes.c_int64)]


class PagePlan(NamedTuple):
    """What page_plan leaves for the step (device tensors; info is int64 [4]:
    status (PLAN_STATUS), tokens, pages taken, first free entry after them)."""
    cu_new: torch.Tensor
    kv_len: torch.Tensor
    slot_map: torch.Tensor
    positions: torch.Tensor
    info: torch.Tensor


class TreePlan(NamedTuple):
    """What tree_plan leaves for the step (device tensors)."""
    positions: torch.Tensor
    mask: torch.Tensor


class Cache(ctypes.Structure):
    """rsa_cache."""
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("dt", ctypes.c_int), ("layers", ctypes.c_int),
                ("n_pages", ctypes.c_int64), ("Hkv", ctypes.c_int), ("page_size", ctypes.c_int), ("d", ctypes.c_int)]


_p, _i32, _i64, _size = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
SIGS = {
    "rsa_page_plan": [_p, _p, _i32, _i32, _i64, _p, _i64, _i32, _p, _i64, _p, _i64, _i64, _p, _p, _p, _p, _p, _p],
    "rsa_qk_norm_rope_fwd": [_p, Heads, Heads, Heads, _p, _p, _p, _i32, _i64, _p],
    "rsa_qk_norm_rope_bwd_workspace_size": [_i32, ctypes.POINTER(_size)],
    "rsa_qk_norm_rope_bwd": [_p, Heads, Heads, Heads, Heads, _p, _p, _p, _size, _p],
    "rsa_prefix_attn_workspace_size": [_i32, _i64, _i32, _i32, _i32, _i32, ctypes.POINTER(_size)],
    "rsa_prefix_attn_fwd": [_p, _i64, _i64, _p, _p, _i32, _i64, _i32, _i32, _i32, _i32, _i64, _p, _p, _i32, _p, _i64, _i32,
                            _p, _i64, _p, _p, _p, _size, _p],
    "rsa_tree_plan": [_p, _i64, _p, _p, _i32, _i32, _i64, _p, _p, _p],
    "rsa_tree_attn_fwd": [_p, _i64, _i64, _p, _p, _i32, _i64, _i32, _i32, _i32, _i32, _i64, _p, _p, _i32, _p, _i64, _i32,
                          _p, _i64, _p, _i64, _i32, _p, _p, _p, _size, _p],
    "rsa_tree_attn_workspace_size": [_i32, _i64, _i32, _i32, _i32, _i32, ctypes.POINTER(_size)],
    "rsa_cache_compact": [_p, _p, _i64, _i32, _p, _p, _i32, _p, _i64, _i32, _p, _p, _p],
    "rsa_page_fork": [_p, _p, _i64, _i32, _p, _i32, _p, _p, _i32, _p, _i64, _p, _p, _p, _p],
    "rsa_page_free": [_p, _i64, _i32, _p, _p, _i32, _i32, _i64, _p, _i64, _p, _p, _p, _p],
}

_DT = {torch.float32: RSA_F32, torch.bfloat16: RSA_BF16}


_native = None
_native_lock = threading.Lock()


def _share(stream, index: int, tensors) -> None:
    """Tensors made on the device's current stream that a call on `stream` uses."""
    stream.wait_stream(torch.cuda.current_stream(index))
    for t in tensors:
        t.record_stream(stream)


def _load_native():
    """The extension module, built first if it is stale, on the loaded librsa."""
    global _native
    with _native_lock:
        if _native is None:
            lib, path = load(), _build.build_binding()
            spec = importlib.util.spec_from_loader("_paged", importlib.machinery.ExtensionFileLoader("_paged", path))
            m = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(m)
            m.bind(*(ctypes.cast(getattr(lib, n), _p).value for n in (
                "rsa_page_plan", "rsa_qk_norm_rope_fwd", "rsa_qk_norm_rope_bwd", "rsa_qk_norm_rope_bwd_workspace_size",
                "rsa_prefix_attn_fwd", "rsa_prefix_attn_workspace_size", "rsa_tree_plan", "rsa_tree_attn_fwd", "rsa_cache_compact",
                "rsa_page_fork", "rsa_page_free", "rsa_tree_attn_workspace_size")), _share)
            _native = m
    return _native


def _error(fn: str, status: int) -> RsaError:
    detail = load().rsa_last_error_string()
    return RsaError(fn, status, detail.decode() if detail else "")


def page_plan(cached_len: torch.Tensor, new_len: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
              page_size: int, n_pages: int, max_tokens: int, free_start: Optional[torch.Tensor] = None, pos0: int = 0,
              out: Optional[PagePlan] = None, stream=None) -> PagePlan:
    """One step's plan from the requests' lengths (rsa_page_plan): fresh pages
    from free_pages [n] int32, from entry free_start[0] (int64 [1]) on, are
    appended to block_table [R, max_pages] int32 in place; each of the new
    tokens gets its cache slot and position, rows behind them slot -1.
    cached_len and new_len are int32 [R].  Check info[0] (PLAN_STATUS) where the
    host can afford to wait: a step that cannot be planned changes nothing."""
    r = (_native or _load_native()).page_plan(cached_len, new_len, block_table, free_pages, page_size, n_pages, max_tokens,
                                              free_start, pos0, out, stream)
    if r.__class__ is int:
        raise _error("rsa_page_plan", r)
    return PagePlan._make(r) if out is None else out


def qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, eps: float = 1e-6, interleaved: bool = False,
                 sections: Optional[Sequence[int]] = None, v=None, slot_map=None, k_cache=None, v_cache=None,
                 q_out=None, k_out=None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """RMS norm of every head of q [T, Hq, d] and k [T, Hkv, d], then the
    rotation by the tokens' positions (rsa_qk_norm_rope_fwd).  cos_sin
    [max_pos, rot] fp32 (rope_table makes it; None: no rotation); positions
    int64 [T], or [axes, T] with `sections` frequencies for each axis.  With
    slot_map [T] int64, k's results and v's rows go to their slots of k_cache
    and v_cache [n_pages, Hkv, page_size, d].  Returns (q_out, k_out); k_out is
    None if it is not given and there is a cache.  q_out may be q and k_out k."""
    r = (_native or _load_native()).qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, sections, v,
                                                 slot_map, k_cache, v_cache, q_out, k_out, stream)
    if r.__class__ is int:
        raise _error("rsa_qk_norm_rope_fwd", r)
    return r


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions, cos_sin, eps: float = 1e-6,
                     interleaved: bool = False, sections: Optional[Sequence[int]] = None, dq=None, dk=None,
                     workspace=None, stream=None, dq_weight=None, dk_weight=None):
    """Gradients of qk_norm_rope (rsa_qk_norm_rope_bwd) from those of its
    results: (dq, dk in q's dtype, dq_weight, dk_weight fp32 [d], None for a
    weight that is None).  dq may be dq_out or q, and dk dk_out or k; dq,
    dk, dq_weight and dk_weight are made if they are not given."""
    r = (_native or _load_native()).qk_norm_rope_bwd(q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, sections,
                                                     dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace, stream)
    if r.__class__ is int:
        raise _error("rsa_qk_norm_rope_bwd", r)
    return r


def rope_table(max_pos: int, rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """cos_sin [max_pos, rot] fp32 for qk_norm_rope: frequency i turns by
    pos * base^(-2i / rot).  The angles are taken in 64 bits (a far position's
    would lose their fraction in 32)."""
    half = rot // 2
    freq = base ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    ang = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def _workspace_size(fn: str, dtype: torch.dtype, *shape: int) -> int:
    n = ctypes.c_size_t(0)
    lib = load()
    st = getattr(lib, fn)(_DT.get(dtype, -1), *shape, ctypes.byref(n))
    if st != 0:
        raise RsaError(fn, st, lib.rsa_last_error_string().decode())
    return int(n.value)


def prefix_attn_workspace_size(dtype: torch.dtype, T: int, Hq: int, Hkv: int, d: int, R: int) -> int:
    return _workspace_size("rsa_prefix_attn_workspace_size", dtype, T, Hq, Hkv, d, R)


def prefix_attn(q, k_cache, v_cache, cu_q, block_table, kv_len, prefix_pages=None, prefix_len: int = 0, out=None,
                lse=None, workspace=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of the step's rows q [T, Hq, d] over a prefix that all requests
    share (tokens [0, prefix_len) in pages prefix_pages) and each request's own
    kv_len[r] tokens in the pages of its row of block_table
    (rsa_prefix_attn_fwd).  Request r's rows [cu_q[r], cu_q[r + 1]) are its
    newest tokens.  Returns (out [T, Hq, d], lse [T, Hq] fp32); rows from
    cu_q[R] on are left as they were.  Calls that may run at the same time need
    workspaces of their own (prefix_attn_workspace_size bytes)."""
    r = (_native or _load_native()).prefix_attn(q, k_cache, v_cache, cu_q, block_table, kv_len, prefix_pages, prefix_len, out, lse,
                                                workspace, stream)
    if r.__class__ is int:
        raise _error("rsa_prefix_attn_fwd", r)
    return r


def tree_plan(parent: torch.Tensor, cu_new: torch.Tensor, kv_len: torch.Tensor, max_tree: int, pos0: int = 0,
              out: Optional[TreePlan] = None, stream=None) -> TreePlan:
    """Positions and ancestor masks of a step's drafted tokens (rsa_tree_plan).
    parent [T] int32: for each row of the step (page_plan's, cu_new and kv_len with
    it) the index of the token's parent among its request's new tokens, -1 for one that
    follows the cached tokens; a token comes after its parent.  max_tree: the most
    drafted tokens of a request, up to 1024.  positions int64 [T] take the place of
    page_plan's; mask int32 [T, ceil(max_tree / 32)] is for tree_attn."""
    r = (_native or _load_native()).tree_plan(parent, cu_new, kv_len, max_tree, pos0, out, stream)
    if r.__class__ is int:
        raise _error("rsa_tree_plan", r)
    return TreePlan._make(r) if out is None else out


def tree_attn(q, k_cache, v_cache, cu_q, block_table, kv_len, tree_mask, prefix_pages=None, prefix_len: int = 0, out=None,
              lse=None, workspace=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """prefix_attn for drafted tokens (rsa_tree_attn_fwd): row i of request r's n
    sees the prefix, the request's own tokens before its drafted ones, and those of
    its drafted tokens j <= i whose bit (bit j mod 32 of word j // 32) is set in the
    row of tree_mask, int32 [T, words]; the mask is tree_plan's or the caller's
    own.  workspace: tree_attn_workspace_size bytes."""
    r = (_native or _load_native()).tree_attn(q, k_cache, v_cache, cu_q, block_table, kv_len, tree_mask, prefix_pages, prefix_len, out,
                                              lse, workspace, stream)
    if r.__class__ is int:
        raise _error("rsa_tree_attn_fwd", r)
    return r


def tree_attn_workspace_size(dtype: torch.dtype, T: int, Hq: int, Hkv: int, d: int, R: int) -> int:
    return _workspace_size("rsa_tree_attn_workspace_size", dtype, T, Hq, Hkv, d, R)


def cache_compact(k_cache, v_cache, block_table, cached_len, kv_len, keep, keep_len, out=None, stream=None) -> torch.Tensor:
    """Keeps some of each request's newest tokens and closes the gaps
    (rsa_cache_compact): own token cached_len[r] + i takes the rows of own token
    cached_len[r] + keep[r, i], i < keep_len[r], in every layer of k_cache and v_cache
    [n_pages, Hkv, page_size, d] or [layers, n_pages, Hkv, page_size, d].  keep
    [R, max_keep] int32, strictly ascending in a row's first keep_len[r] entries.
    Returns the new lengths, int32 [R]: cached_len + keep_len.  Keys keep their rotation:
    where cached tokens are dropped, later positions go on behind theirs (see the module).
    The pages must be the request's own: one that shares some is forked with shares=None first."""
    r = (_native or _load_native()).cache_compact(k_cache, v_cache, block_table, cached_len, kv_len, keep, keep_len, out, stream)
    if r.__class__ is int:
        raise _error("rsa_cache_compact", r)
    return r[0]


def page_fork(k_cache, v_cache, block_table, kv_len, src, dst, free_pages, free_start: Optional[torch.Tensor] = None, shares=None,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Request dst[f] becomes a copy of request src[f] (rsa_page_fork): with shares
    [n_pages] int32 (users of a page beyond the first; zeros to begin with) full
    pages are shared and the partial last one is copied, without every page is.
    block_table, kv_len and shares are updated in place, rows are copied in every layer
    of the caches (as in cache_compact; a fork is one call, with all layers); fresh pages come from free_pages as in
    page_plan.  Returns info, int64 [4]: status (PLAN_STATUS), entries shared, pages
    taken, first free entry after them.  Forks that cannot all be made change nothing; an entry
    with -1 in both lists is no fork, so that a captured call may make any number up to its own."""
    r = (_native or _load_native()).page_fork(k_cache, v_cache, block_table, kv_len, src, dst, free_pages, free_start, shares, out, stream)
    if r.__class__ is int:
        raise _error("rsa_page_fork", r)
    return r[0]


def page_free(block_table, kv_len, keep_len, free_pages, free_start: torch.Tensor, page_size: int, n_pages: int, shares=None,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Requests keep their first keep_len [R] of kv_len tokens (0: the request ends)
    and give the pages behind them back (rsa_page_free): those without another user,
    by shares if given, go to free_pages before entry free_start[0], ascending.  Returns
    info, int64 [4]: status (PLAN_STATUS), pages freed, entries given back, the new
    free_start.  What cannot all be given back changes nothing."""
    r = (_native or _load_native()).page_free(block_table, kv_len, keep_len, free_pages, free_start, page_size, n_pages, shares, out, stream)
    if r.__class__ is int:
        raise _error("rsa_page_free", r)
    return r[0]
