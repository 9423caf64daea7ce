"""Serving over a paged KV cache: a step's plan, the norm and rotation of its
heads with the cache write, and attention behind a shared prefix.

The calls of ``include/rsa.h`` with the same names; as in the rest of the
binding they only check and marshal arguments, here in an extension module
(csrc/torch_paged.cpp), as a step makes many of them.  One decode step:

    plan = page_plan(cached_len, new_len, block_table, free_pages, page_size, n_pages, max_tokens, pos0=prefix_len)
    for each layer:
        q, _ = qk_norm_rope(q, k, wq, wk, plan.positions, cos_sin, v=v, slot_map=plan.slot_map,
                            k_cache=k_cache, v_cache=v_cache)
        out, lse = prefix_attn(q, k_cache, v_cache, plan.cu_new, block_table, plan.kv_len,
                               prefix_pages=prefix_pages, prefix_len=prefix_len)

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
               4: "more tokens than max_tokens"}


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


_p, _i32, _i64, _size = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
SIGS = {
    "rsa_page_plan": [_p, _p, _i32, _i32, _i64, _p, _i64, _i32, _p, _i64, _p, _i64, _i64, _p, _p, _p, _p, _p, _p],
    "rsa_qk_norm_rope_fwd": [_p, Heads, Heads, Heads, _p, _p, _p, _i32, _i64, _p],
    "rsa_qk_norm_rope_bwd_workspace_size": [_i32, ctypes.POINTER(_size)],
    "rsa_qk_norm_rope_bwd": [_p, Heads, Heads, Heads, Heads, _p, _p, _p, _size, _p],
    "rsa_prefix_attn_workspace_size": [_i32, _i64, _i32, _i32, _i32, _i32, ctypes.POINTER(_size)],
    "rsa_prefix_attn_fwd": [_p, _i64, _i64, _p, _p, _i32, _i64, _i32, _i32, _i32, _i32, _i64, _p, _p, _i32, _p, _i64, _i32,
                            _p, _i64, _p, _p, _p, _size, _p],
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
                "rsa_prefix_attn_fwd", "rsa_prefix_attn_workspace_size")), _share)
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


def prefix_attn_workspace_size(dtype: torch.dtype, T: int, Hq: int, Hkv: int, d: int, R: int) -> int:
    n = ctypes.c_size_t(0)
    lib = load()
    st = lib.rsa_prefix_attn_workspace_size(_DT.get(dtype, -1), T, Hq, Hkv, d, R, ctypes.byref(n))
    if st != 0:
        raise RsaError("rsa_prefix_attn_workspace_size", st, lib.rsa_last_error_string().decode())
    return int(n.value)


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
