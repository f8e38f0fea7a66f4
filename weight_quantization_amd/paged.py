"""ctypes binding of libhlwq's serving operators (declared in include/hlwq_attention.h).

A paged KV cache of HLWQ codes: page planning, append and attention, and the
attention over whole prompts that precedes them.  One step of a generation loop:

    plan = hlwq_kv_page_plan(tokens, n_new, free_pages, n_free, block_table, rows)
    out = hlwq_kv_paged_attention(q, k, v, plan.cu_new, plan.lens, block_table, *cache)
    hlwq_kv_paged_append(k, v, plan.cu_new, plan.lens, plan.row_request, plan.slots, *cache)
    tokens, n_free = plan.lens, plan.n_free

with cache = (k_packed, k_norms, v_packed, v_norms, k_window, v_window).  As in
``binding``, every function checks its tensors, passes pointers, sizes and the
current stream to the C function of the same name and raises on a status.
"""
from __future__ import annotations

import ctypes
import math
from typing import TYPE_CHECKING, NamedTuple

from . import binding
from .binding import KV_DIM, _check, _i64, _int, _ptr, _stream_handle, _torch, _vp, load_library

if TYPE_CHECKING:
    import torch


class KvStore(ctypes.Structure):
    _fields_ = [("packed", _vp), ("norms", _vp), ("window", _vp)]


class KvCache(ctypes.Structure):
    _fields_ = [("k", KvStore), ("v", KvStore), ("n_pages", _i64), ("requests", _i64), ("kv_heads", _i64),
                ("page_size", _i64), ("n_residual", _i64), ("ring", _i64), ("head_dim", _int), ("bits", _int)]


class KvPlanArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("tokens", "n_new", "reset", "n_free", "free_pages", "block_table", "cu_new", "lens",
                                   "row_request", "positions", "slots", "n_free_after", "status")]
    _fields_ += [(n, _i64) for n in ("requests", "rows", "max_pages", "n_pages", "page_size", "n_residual")]


binding._SIGNATURES.update({
    "hlwq_kv_page_plan": (_int, [ctypes.POINTER(KvPlanArgs), _vp]),
    "hlwq_kv_paged_append": (_int, [ctypes.POINTER(KvCache), _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp]),
    "hlwq_kv_paged_attention": (_int, [ctypes.POINTER(KvCache), _vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp,
                                       _i64, _i64, ctypes.c_float, _vp, _vp, ctypes.c_size_t, _vp]),
    "hlwq_kv_paged_attention_workspace": (ctypes.c_size_t, [_i64, _i64, _i64, _i64]),
    "hlwq_prompt_attention": (_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _int, ctypes.c_float,
                                     _vp, _vp]),
})


class KvPagePlan(NamedTuple):
    """What hlwq_kv_page_plan writes, int32 on the device."""
    cu_new: torch.Tensor       # [requests + 1] prefix sum of the step's tokens
    lens: torch.Tensor         # [requests] tokens after the step
    row_request: torch.Tensor  # [rows]
    positions: torch.Tensor    # [rows]
    slots: torch.Tensor        # [rows]
    n_free: torch.Tensor       # [1] free pages after the step
    status: torch.Tensor       # [1] 0, the number of missing pages, or -1


def _empty(shape, dtype, device, stream):
    """A new tensor that the call's stream uses first: the allocator hands memory out in the order of one stream."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _buf(t, dtype, shape, name):
    """A contiguous device tensor of this type and shape (None: any extent)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be in device memory")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    s = t.shape
    if len(s) != len(shape) or any(w is not None and g != w for g, w in zip(s, shape)):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(s)}")
    return t


def _rows(t, heads, name):
    """Token rows [rows, heads, 256] in bf16: whole head vectors side by side, any row stride that is a multiple
    of 8 (a slice of a fused projection's output will do).  Returns the row stride in elements."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be in device memory")
    s = t.shape
    if len(s) != 3 or s[2] != KV_DIM or (heads is not None and s[1] != heads):
        raise ValueError(f"{name} must be [rows, {'heads' if heads is None else heads}, {KV_DIM}], got {list(s)}")
    row, head, one = t.stride()
    if t.numel() == 0 or s[0] == 1:
        row = max(row, s[1] * KV_DIM)
        row += -row % 8
    if t.numel() and (one != 1 or (s[1] > 1 and head != KV_DIM) or row < s[1] * KV_DIM or row % 8):
        raise ValueError(f"{name} must hold each row's heads side by side, rows a multiple of 8 elements apart; "
                         f"its strides are {t.stride()}")
    return row


def _cache(k_packed, k_norms, v_packed, v_norms, k_window, v_window, requests, n_residual, bits):
    torch = _torch()
    if bits not in (2, 3):
        raise ValueError("bits must be 3 or 2")
    _buf(k_packed, torch.uint8, (None, None, None, 32 * bits), "k_packed")
    pages, heads, page, _ = k_packed.shape
    _buf(v_packed, torch.uint8, (pages, heads, page, 32 * bits), "v_packed")
    _buf(k_norms, torch.float16, (pages, heads, page), "k_norms")
    _buf(v_norms, torch.float16, (pages, heads, page), "v_norms")
    ring = 0
    if k_window is not None or v_window is not None or n_residual:
        _buf(k_window, torch.bfloat16, (requests, heads, None, KV_DIM), "k_window")
        ring = k_window.shape[2]
        _buf(v_window, torch.bfloat16, (requests, heads, ring, KV_DIM), "v_window")
    return KvCache(KvStore(_ptr(k_packed), _ptr(k_norms), _ptr(k_window)),
                   KvStore(_ptr(v_packed), _ptr(v_norms), _ptr(v_window)),
                   pages, requests, heads, page, n_residual, ring, KV_DIM, bits), heads


def hlwq_kv_page_plan(tokens, n_new, free_pages, n_free, block_table, rows: int, page_size: int = 64,
                      n_residual: int = 128, reset=None, stream=None) -> KvPagePlan:
    """Plan one step of a batch: tokens, n_new int32 [requests] (held and new tokens), free_pages int32 [n_pages] (the
    stack of free page ids, n_free int32 [1] of them), block_table int32 [requests, max_pages]; rows: rows of the
    step's tensors, at least the sum of n_new (rows past it are padding); reset uint8 [requests]: nonzero where the
    slot's request has ended, whose pages go back first.  free_pages and block_table are updated in place."""
    torch = _torch()
    _buf(tokens, torch.int32, (None,), "tokens")
    n = tokens.shape[0]
    _buf(n_new, torch.int32, (n,), "n_new")
    _buf(free_pages, torch.int32, (None,), "free_pages")
    _buf(n_free, torch.int32, (1,), "n_free")
    _buf(block_table, torch.int32, (n, None), "block_table")
    if reset is not None:
        _buf(reset, torch.uint8, (n,), "reset")
    if rows < 0:
        raise ValueError("rows must not be negative")
    out = _empty(2 * n + 3 + 3 * rows, torch.int32, tokens.device, stream)
    plan = KvPagePlan(*out.split_with_sizes([n + 1, n, rows, rows, rows, 1, 1]))
    at = out.data_ptr()
    ends = [at + 4 * k for k in (0, n + 1, 2 * n + 1, 2 * n + 1 + rows, 2 * n + 1 + 2 * rows, 2 * n + 1 + 3 * rows,
                                 2 * n + 2 + 3 * rows)]
    args = KvPlanArgs(_ptr(tokens), _ptr(n_new), _ptr(reset), _ptr(n_free), _ptr(free_pages), _ptr(block_table), *ends,
                      n, rows, block_table.shape[1], free_pages.shape[0], page_size, n_residual)
    st = load_library().hlwq_kv_page_plan(
        ctypes.byref(args), _stream_handle(stream, tokens, n_new, free_pages, n_free, block_table, reset))
    _check("hlwq_kv_page_plan", st)
    return plan


def hlwq_kv_paged_append(k_new, v_new, cu_new, lens, row_request, slots, k_packed, k_norms, v_packed, v_norms,
                         k_window, v_window, n_residual: int = 128, bits: int = 3, stream=None):
    """Put a step's keys and values, bf16 [rows, kv_heads, 256] each, into a paged cache: packed uint8
    [n_pages, kv_heads, page_size, 32 * bits], norms fp16 [n_pages, kv_heads, page_size], windows bf16
    [requests, kv_heads, ring, 256] (None when n_residual = 0); cu_new, lens, row_request, slots from the plan."""
    torch = _torch()
    _buf(lens, torch.int32, (None,), "lens")
    n = lens.shape[0]
    cache, heads = _cache(k_packed, k_norms, v_packed, v_norms, k_window, v_window, n, n_residual, bits)
    ks = _rows(k_new, heads, "k_new")
    rows = k_new.shape[0]
    vs = _rows(v_new, heads, "v_new")
    _same_rows(rows, v_new, "v_new")
    _buf(cu_new, torch.int32, (n + 1,), "cu_new")
    _buf(row_request, torch.int32, (rows,), "row_request")
    _buf(slots, torch.int32, (rows,), "slots")
    st = load_library().hlwq_kv_paged_append(
        ctypes.byref(cache), _ptr(k_new), ks, _ptr(v_new), vs, _ptr(cu_new), _ptr(lens), _ptr(row_request), _ptr(slots),
        rows, _stream_handle(stream, k_new, v_new, cu_new, lens, row_request, slots, k_packed, k_norms, v_packed, v_norms,
                             k_window, v_window))
    _check("hlwq_kv_paged_append", st)


def _same_rows(rows, t, name):
    if t.shape[0] != rows:
        raise ValueError(f"{name} must have {rows} rows, got {t.shape[0]}")


def _heads(q, kv_heads):
    if q.shape[1] and (not kv_heads or q.shape[1] % kv_heads):
        raise ValueError(f"{q.shape[1]} query heads do not divide over {kv_heads} KV heads")


def hlwq_kv_paged_attention_workspace(requests: int, rows: int, q_heads: int, kv_heads: int) -> int:
    """Bytes of workspace that hlwq_kv_paged_attention needs for these sizes."""
    return int(load_library().hlwq_kv_paged_attention_workspace(requests, rows, q_heads, kv_heads))


def hlwq_kv_paged_attention(q, k_new, v_new, cu_new, lens, block_table, k_packed, k_norms, v_packed, v_norms,
                            k_window, v_window, n_residual: int = 128, bits: int = 3, scale: float | None = None,
                            out=None, workspace=None, stream=None):
    """Attention of a step's rows (before its append) over pages, window and the step itself: q bf16
    [rows, q_heads, 256], k_new and v_new bf16 [rows, kv_heads, 256], cu_new and lens from the plan, block_table int32
    [requests, max_pages], the cache as in hlwq_kv_paged_append; scale 1 / 16 by default.  Returns bf16
    [rows, q_heads, 256]; rows past cu_new[requests] are left as they were (undefined in a new `out`).  workspace:
    uint8, hlwq_kv_paged_attention_workspace bytes; allocated for the call by default."""
    torch = _torch()
    _buf(lens, torch.int32, (None,), "lens")
    n = lens.shape[0]
    cache, heads = _cache(k_packed, k_norms, v_packed, v_norms, k_window, v_window, n, n_residual, bits)
    qs = _rows(q, None, "q")
    rows, q_heads, _ = q.shape
    _heads(q, heads)
    ks, vs = _rows(k_new, heads, "k_new"), _rows(v_new, heads, "v_new")
    _same_rows(rows, k_new, "k_new")
    _same_rows(rows, v_new, "v_new")
    _buf(cu_new, torch.int32, (n + 1,), "cu_new")
    _buf(block_table, torch.int32, (n, None), "block_table")
    if out is None:
        out = _empty((rows, q_heads, KV_DIM), torch.bfloat16, q.device, stream)
    else:
        _buf(out, torch.bfloat16, (rows, q_heads, KV_DIM), "out")
    lib = load_library()
    if workspace is None:
        workspace = _empty(lib.hlwq_kv_paged_attention_workspace(n, rows, q_heads, heads), torch.uint8, q.device, stream)
    else:
        _buf(workspace, torch.uint8, (None,), "workspace")
    st = lib.hlwq_kv_paged_attention(
        ctypes.byref(cache), _ptr(q), qs, q_heads, _ptr(k_new), ks, _ptr(v_new), vs, _ptr(cu_new), _ptr(lens),
        _ptr(block_table), block_table.shape[1], rows, 1 / math.sqrt(KV_DIM) if scale is None else scale, _ptr(out),
        _ptr(workspace), workspace.numel(),
        _stream_handle(stream, q, k_new, v_new, cu_new, lens, block_table, k_packed, k_norms, v_packed, v_norms, k_window,
                       v_window, out, workspace))
    _check("hlwq_kv_paged_attention", st)
    return out


def hlwq_prompt_attention(q, k, v, cu_seqlens, scale: float | None = None, out=None, stream=None):
    """Causal attention over whole prompts packed one after the other: q bf16 [rows, q_heads, 256], k and v bf16
    [rows, kv_heads, 256], cu_seqlens int32 [sequences + 1]; scale 1 / 16 by default.  Returns bf16
    [rows, q_heads, 256]; rows past cu_seqlens[-1] are left as they were (undefined in a new `out`)."""
    torch = _torch()
    qs = _rows(q, None, "q")
    rows, q_heads, _ = q.shape
    ks = _rows(k, None, "k")
    heads = k.shape[1]
    _heads(q, heads)
    vs = _rows(v, heads, "v")
    _same_rows(rows, k, "k")
    _same_rows(rows, v, "v")
    _buf(cu_seqlens, torch.int32, (None,), "cu_seqlens")
    if cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must have at least one entry")
    if out is None:
        out = _empty((rows, q_heads, KV_DIM), torch.bfloat16, q.device, stream)
    else:
        _buf(out, torch.bfloat16, (rows, q_heads, KV_DIM), "out")
    st = load_library().hlwq_prompt_attention(
        _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(cu_seqlens), cu_seqlens.shape[0] - 1, rows, q_heads, heads, KV_DIM,
        1 / math.sqrt(KV_DIM) if scale is None else scale, _ptr(out), _stream_handle(stream, q, k, v, cu_seqlens, out))
    _check("hlwq_prompt_attention", st)
    return out
