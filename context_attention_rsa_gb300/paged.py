"""Serving over a paged KV cache: a step's plan, the norm and rotation of its
heads with the cache write, and attention behind a shared prefix.

The calls of ``include/rsa.h`` with the same names; as in the rest of the
binding they only check and marshal arguments.  One decode step:

    plan = page_plan(cached_len, new_len, block_table, free_pages, page_size, n_pages, max_tokens, pos0=prefix_len)
    for each layer:
        q, _ = qk_norm_rope(q, k, wq, wk, plan.positions, cos_sin, v=v, slot_map=plan.slot_map,
                            k_cache=k_cache, v_cache=v_cache)
        out, lse = prefix_attn(q, k_cache, v_cache, plan.cu_new, block_table, plan.kv_len,
                               prefix_pages=prefix_pages, prefix_len=prefix_len)

Caches are [n_pages, Hkv, page_size, d]; a step's rows are packed [T, H, d].
Nothing synchronises, so a step can be captured into a CUDA graph and replayed
with other lengths: what depends on them is read on the device.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import RSA_BF16, RSA_F32, RsaError, load

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
# NormRopeArgs as one packed record (native alignment): filling the ctypes fields one by
# one cost more than the launch.
_NORM_ROPE = struct.Struct("@iqiiiPqqPqqPPfiiiiiiiPPq")
assert _NORM_ROPE.size == ctypes.sizeof(NormRopeArgs)

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


def _dtype(t: torch.Tensor) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")
    return dt


def _check(name: str, t, dim: int, dtype: torch.dtype, device: torch.device, contiguous: bool = True) -> None:
    try:
        if t.dtype is dtype and t.dim() == dim and t.device == device and (not contiguous or t.is_contiguous()):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device:
        raise TypeError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype != dtype or t.dim() != dim:
        raise ValueError(f"{name} must be a {dim}-d {dtype} tensor (got {t.dim()}-d {t.dtype})")
    raise ValueError(f"{name} must be contiguous")


def _row_layout(name: str, t, dtype: torch.dtype, device: torch.device, shape=None) -> Tuple[int, int, int]:
    """Address, token and head stride of a [T, H, d] operand."""
    _check(name, t, 3, dtype, device, contiguous=False)
    T, H, d = t.shape
    if shape is not None and (T, H, d) != shape:
        raise ValueError(f"{name} must be {tuple(shape)} (got {(T, H, d)})")
    ts, hs, es = t.stride()
    if es != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    # the stride of a dimension of one says nothing: put the dense one in its place
    if H == 1:
        hs = d
    if T == 1:
        ts = H * hs
    return t.data_ptr(), ts, hs


def _heads(name: str, t, dtype: torch.dtype, device: torch.device, shape=None) -> Heads:
    return Heads(*_row_layout(name, t, dtype, device, shape))


def _new_rows(shape, dtype: torch.dtype, device: torch.device, made: list) -> Tuple[torch.Tensor, Heads]:
    """A dense [T, H, d] result."""
    t = torch.empty(shape, dtype=dtype, device=device)
    made.append(t)
    return t, Heads(t.data_ptr(), shape[1] * shape[2], shape[2])


# The device's current stream as a bare handle (a Stream object takes longer to make than a launch).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call_on(device: torch.device, fn: str, stream, temporaries: Sequence[torch.Tensor], *args) -> None:
    """The library's call on `device` and `stream` (default: the device's current stream)."""
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call_on(device, fn, stream, temporaries, *args)
    handle = _raw_stream(index)
    if stream is not None:
        if hasattr(stream, "cuda_stream"):
            if temporaries and stream.cuda_stream != handle:
                # made on the current stream, used on another one: their memory may still be in use
                # there, and is not to be handed out again before the call is done
                stream.wait_stream(torch.cuda.current_stream(index))
                for t in temporaries:
                    t.record_stream(stream)
            handle = stream.cuda_stream
        elif temporaries and handle != int(stream):
            raise ValueError("with a bare stream handle other than the current stream's, pass every output and workspace")
        else:
            handle = int(stream)
    lib = load()
    st = getattr(lib, fn)(*args, handle)
    if st != 0:
        detail = lib.rsa_last_error_string()
        raise RsaError(fn, st, detail.decode() if detail else "")


def _workspace(n: int, device: torch.device, stream, made: list) -> Tuple[int, int]:
    """Address and bytes of device memory for one call, kept by `made` until it is enqueued."""
    if stream is None:
        # (after a launch a tensor costs 2 to 4 us more to make than its memory)
        made.append(torch.UntypedStorage(n, device=device))
    else:
        made.append(torch.empty(n, dtype=torch.uint8, device=device))  # (can be recorded on another stream)
    return made[-1].data_ptr(), n


def page_plan(cached_len: torch.Tensor, new_len: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
              page_size: int, n_pages: int, max_tokens: int, free_start: Optional[torch.Tensor] = None, pos0: int = 0,
              out: Optional[PagePlan] = None, stream=None) -> PagePlan:
    """One step's plan from the requests' lengths (rsa_page_plan): fresh pages
    from free_pages [n] int32, from entry free_start[0] (int64 [1]) on, are
    appended to block_table [R, max_pages] int32 in place; each of the new
    tokens gets its cache slot and position, rows behind them slot -1.
    cached_len and new_len are int32 [R].  Check info[0] (PLAN_STATUS) where the
    host can afford to wait: a step that cannot be planned changes nothing."""
    if not isinstance(cached_len, torch.Tensor) or not cached_len.is_cuda:
        raise TypeError("cached_len must be a CUDA tensor")
    dev = cached_len.device
    _check("cached_len", cached_len, 1, torch.int32, dev)
    R = cached_len.shape[0]
    _check("new_len", new_len, 1, torch.int32, dev)
    _check("block_table", block_table, 2, torch.int32, dev, contiguous=False)
    _check("free_pages", free_pages, 1, torch.int32, dev)
    if new_len.shape[0] != R or block_table.shape[0] != R:
        raise ValueError("new_len and block_table must have cached_len's requests")
    max_pages = block_table.shape[1]
    if block_table.stride(1) != 1 and max_pages > 1:
        raise ValueError("rows of block_table must be contiguous")
    if free_start is not None:
        _check("free_start", free_start, 1, torch.int64, dev)
        if free_start.shape[0] < 1:
            raise ValueError("free_start must hold one entry")
    made = ()
    if out is None:
        i32, i64 = torch.int32, torch.int64
        out = made = PagePlan(torch.empty(R + 1, dtype=i32, device=dev), torch.empty(R, dtype=i32, device=dev),
                              torch.empty(max_tokens, dtype=i64, device=dev), torch.empty(max_tokens, dtype=i64, device=dev),
                              torch.empty(4, dtype=i64, device=dev))
    else:
        for name, t, n, dt in (("cu_new", out.cu_new, R + 1, torch.int32), ("kv_len", out.kv_len, R, torch.int32),
                               ("slot_map", out.slot_map, max_tokens, torch.int64),
                               ("positions", out.positions, max_tokens, torch.int64), ("info", out.info, 4, torch.int64)):
            _check("out." + name, t, 1, dt, dev)
            if t.shape[0] != n:
                raise ValueError(f"out.{name} must hold {n} entries")
    _call_on(dev, "rsa_page_plan", stream, made, cached_len.data_ptr(), new_len.data_ptr(), R, page_size, n_pages,
             block_table.data_ptr(), max_pages if R == 1 else block_table.stride(0), max_pages, free_pages.data_ptr(),
             free_pages.shape[0], None if free_start is None else free_start.data_ptr(), pos0, max_tokens,
             out.cu_new.data_ptr(), out.kv_len.data_ptr(), out.slot_map.data_ptr(), out.positions.data_ptr(),
             out.info.data_ptr())
    return out


def _norm_rope_args(q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, sections) -> bytes:
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3:
        raise TypeError("q must be a CUDA tensor [T, Hq, d]")
    dev, dt = q.device, q.dtype
    code = _dtype(q)
    T, Hq, d = q.shape
    q_at, k_at = _row_layout("q", q, dt, dev), _row_layout("k", k, dt, dev)
    if k.shape[0] != T or k.shape[2] != d:
        raise ValueError("q [T, Hq, d] and k [T, Hkv, d] must agree")
    wq = wk = rot = max_pos = table = pos = 0
    if q_weight is not None:
        _check("q_weight", q_weight, 1, dt, dev)
        wq = q_weight.data_ptr()
    if k_weight is not None:
        _check("k_weight", k_weight, 1, dt, dev)
        wk = k_weight.data_ptr()
    if (wq and q_weight.shape[0] != d) or (wk and k_weight.shape[0] != d):
        raise ValueError(f"q_weight and k_weight must hold d={d} values")
    axes, parts = 1, (0, 0, 0, 0)
    if cos_sin is not None:
        _check("cos_sin", cos_sin, 2, torch.float32, dev)
        max_pos, rot = cos_sin.shape
        table = cos_sin.data_ptr()
        if sections is not None:
            axes = len(sections)
            if not 1 <= axes <= 4:
                raise ValueError("sections must name one to four axes")
            if axes == 1 and sections[0] != rot // 2:
                raise ValueError("one section must hold all rot/2 frequencies")
            parts = (*sections, 0, 0, 0)[:4]
        if not isinstance(positions, torch.Tensor):
            raise TypeError("positions must be a CUDA tensor")
        _check("positions", positions, positions.dim() if axes == 1 else 2, torch.int64, dev)
        if positions.shape[-1] != T or positions.numel() != axes * T:
            raise ValueError(f"positions must be int64 [{axes}, {T}]" if axes > 1 else f"positions must be int64 [{T}]")
        pos = positions.data_ptr()
    return _NORM_ROPE.pack(code, T, Hq, k.shape[1], d, *q_at, *k_at, wq, wk, eps, rot, 1 if interleaved else 0, axes, *parts,
                           pos, table, max_pos)


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
    a = _norm_rope_args(q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, sections)
    dev, dt, q_shape, k_shape = q.device, q.dtype, tuple(q.shape), tuple(k.shape)
    made = []
    if q_out is None:
        q_out, qo = _new_rows(q_shape, dt, dev, made)
    else:
        qo = _heads("q_out", q_out, dt, dev, q_shape)
    if k_out is not None:
        ko = _heads("k_out", k_out, dt, dev, k_shape)
    elif slot_map is None:
        k_out, ko = _new_rows(k_shape, dt, dev, made)
    else:
        ko = Heads()
    if slot_map is None:
        if v is not None or k_cache is not None or v_cache is not None:
            raise ValueError("v, k_cache and v_cache go with slot_map")
        _call_on(dev, "rsa_qk_norm_rope_fwd", stream, made, a, qo, ko, Heads(), None, None, None, 0, 0)
        return q_out, k_out
    _check("slot_map", slot_map, 1, torch.int64, dev)
    if slot_map.shape[0] != q_shape[0]:
        raise ValueError(f"slot_map must hold T={q_shape[0]} slots")
    vh = _heads("v", v, dt, dev, k_shape)
    n_pages, page_size = _check_caches(k_cache, v_cache, k_shape[1], k_shape[2], dt, dev)
    _call_on(dev, "rsa_qk_norm_rope_fwd", stream, made, a, qo, ko, vh, slot_map.data_ptr(), k_cache.data_ptr(),
             v_cache.data_ptr(), page_size, n_pages)
    return q_out, k_out


@functools.lru_cache(maxsize=None)
def _norm_rope_bwd_workspace_size(d: int) -> int:
    n = ctypes.c_size_t(0)
    load().rsa_qk_norm_rope_bwd_workspace_size(d, ctypes.byref(n))
    return n.value or 1  # (the call itself refuses another d)


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions, cos_sin, eps: float = 1e-6,
                     interleaved: bool = False, sections: Optional[Sequence[int]] = None, dq=None, dk=None,
                     workspace=None, stream=None):
    """Gradients of qk_norm_rope (rsa_qk_norm_rope_bwd) from those of its
    results: (dq, dk in q's dtype, dq_weight, dk_weight fp32 [d], None for a
    weight that is None).  dq may be dq_out and dk may be dk_out."""
    a = _norm_rope_args(q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, sections)
    dev, dt, q_shape, k_shape = q.device, q.dtype, tuple(q.shape), tuple(k.shape)
    gq, gk = _heads("dq_out", dq_out, dt, dev, q_shape), _heads("dk_out", dk_out, dt, dev, k_shape)
    made = []
    if dq is None:
        dq, dqh = _new_rows(q_shape, dt, dev, made)
    else:
        dqh = _heads("dq", dq, dt, dev, q_shape)
    if dk is None:
        dk, dkh = _new_rows(k_shape, dt, dev, made)
    else:
        dkh = _heads("dk", dk, dt, dev, k_shape)
    d = q_shape[2]
    dwq = dwk = None
    if q_weight is not None:
        dwq = torch.empty(d, dtype=torch.float32, device=dev)
        made.append(dwq)
    if k_weight is not None:
        dwk = torch.empty(d, dtype=torch.float32, device=dev)
        made.append(dwk)
    if workspace is None:
        ws = _workspace(_norm_rope_bwd_workspace_size(d), dev, stream, made)
    else:
        ws = workspace.data_ptr(), workspace.nbytes
    _call_on(dev, "rsa_qk_norm_rope_bwd", stream, made, a, gq, gk, dqh, dkh, None if dwq is None else dwq.data_ptr(),
             None if dwk is None else dwk.data_ptr(), *ws)
    return dq, dk, dwq, dwk


def rope_table(max_pos: int, rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """cos_sin [max_pos, rot] fp32 for qk_norm_rope: frequency i turns by
    pos * base^(-2i / rot).  The angles are taken in 64 bits (a far position's
    would lose their fraction in 32)."""
    half = rot // 2
    freq = base ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    ang = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def _check_caches(k_cache, v_cache, Hkv: int, d: int, dt: torch.dtype, dev: torch.device) -> Tuple[int, int]:
    _check("k_cache", k_cache, 4, dt, dev)
    _check("v_cache", v_cache, 4, dt, dev)
    n_pages, h, page_size, dd = k_cache.shape
    if v_cache.shape != k_cache.shape or h != Hkv or dd != d:
        raise ValueError(f"k_cache and v_cache must both be [n_pages, Hkv={Hkv}, page_size, d={d}]")
    return n_pages, page_size


@functools.lru_cache(maxsize=1024)
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
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3:
        raise TypeError("q must be a CUDA tensor [T, Hq, d]")
    dev, dt = q.device, q.dtype
    code = _dtype(q)
    T, Hq, d = q.shape
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [n_pages, Hkv, page_size, d]")
    Hkv = k_cache.shape[1]
    n_pages, page_size = _check_caches(k_cache, v_cache, Hkv, d, dt, dev)
    q_at = _row_layout("q", q, dt, dev)
    _check("cu_q", cu_q, 1, torch.int32, dev)
    _check("kv_len", kv_len, 1, torch.int32, dev)
    _check("block_table", block_table, 2, torch.int32, dev, contiguous=False)
    R, max_pages = block_table.shape
    if cu_q.shape[0] != R + 1 or kv_len.shape[0] != R:
        raise ValueError("cu_q [R + 1], kv_len [R] and block_table [R, max_pages] must agree")
    if block_table.stride(1) != 1 and max_pages > 1:
        raise ValueError("rows of block_table must be contiguous")
    if prefix_len:
        _check("prefix_pages", prefix_pages, 1, torch.int32, dev)
        if prefix_pages.shape[0] * page_size < prefix_len:
            raise ValueError(f"prefix_pages hold {prefix_pages.shape[0] * page_size} tokens, prefix_len is {prefix_len}")
    made = []
    if out is None:
        out = torch.empty((T, Hq, d), dtype=dt, device=dev)
        made.append(out)
    else:
        _check("out", out, 3, dt, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
        made.append(lse)
    else:
        _check("lse", lse, 2, torch.float32, dev)
        if lse.shape != q.shape[:2]:
            raise ValueError("lse must be [T, Hq]")
    if workspace is None:
        ws = _workspace(prefix_attn_workspace_size(dt, T, Hq, Hkv, d, R), dev, stream, made)
    else:
        ws = workspace.data_ptr(), workspace.nbytes
    _call_on(dev, "rsa_prefix_attn_fwd", stream, made, *q_at, k_cache.data_ptr(),
             v_cache.data_ptr(), code, T, Hq, Hkv, d, page_size, n_pages, cu_q.data_ptr(), kv_len.data_ptr(), R,
             block_table.data_ptr(), max_pages if R == 1 else block_table.stride(0), max_pages,
             prefix_pages.data_ptr() if prefix_len else None, prefix_len, out.data_ptr(), lse.data_ptr(),
             *ws)
    return out, lse
