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
import struct
from typing import TYPE_CHECKING, NamedTuple

from . import binding
from .binding import KV_DIM, _check, _i64, _int, _stream_handle, _torch, _vp, load_library

if TYPE_CHECKING:
    import torch


binding._SIGNATURES.update({
    "hlwq_kv_page_plan": (_int, [_vp, _vp]),
    "hlwq_kv_paged_append": (_int, [_vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp]),
    "hlwq_kv_paged_attention": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp,
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


# A decode step makes these calls once per layer, so what they cost on the host
# counts: every tensor is checked in one expression, and only a call that is to
# be refused finds out why.

def _fail(t, dtype, name, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be in device memory")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _shape(t, dims, name):
    """The shape of a tensor of this many dimensions."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    s = t.shape
    if len(s) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {list(s)}")
    return s


def _at(t, dtype, shape, name):
    """The address of a contiguous device tensor of this type and shape."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _fail(t, dtype, name, shape)


def _rows(t, rows, heads, bf16, name):
    """Token rows [rows, heads, 256] in bf16: whole head vectors side by side, any row stride that is a multiple
    of 8 (a slice of a fused projection's output will do).  Returns the address and the row stride in elements."""
    try:
        ok = t.dtype is bf16 and t.shape == (rows, heads, KV_DIM) and t.is_cuda
    except AttributeError:
        ok = False
    if not ok:
        s = _shape(t, 3, name)
        if t.dtype is bf16 and t.is_cuda:
            raise ValueError(f"{name} must have {rows} rows of {heads} x {KV_DIM}, got {list(s)}")
        _fail(t, bf16, name)
    row, head, one = t.stride()
    if rows <= 1 or heads == 0:
        row = heads * KV_DIM  # there is no next row
    elif row < heads * KV_DIM or row % 8:
        one = 0
    if (one != 1 or (heads > 1 and head != KV_DIM)) and t.numel():
        raise ValueError(f"{name} must hold each row's heads side by side, rows a multiple of 8 elements apart; "
                         f"its strides are {t.stride()}")
    return t.data_ptr(), row


_one_device = None  # whether the process sees a single device


def _stream(stream, tensors):
    """The stream to launch on (of the current device, as every tensor must be)."""
    global _one_device
    torch = _torch()
    if _one_device is None:
        _one_device = torch.cuda.device_count() == 1
    if stream is None and _one_device:
        return torch.cuda.current_stream().cuda_stream
    return _stream_handle(stream, *tensors)


def _empty(shape, dtype, device, stream):
    """A new tensor that the call's stream uses first: the allocator hands memory out in the order of one stream."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


_CACHE = struct.Struct("6P6q2i")  # hlwq_kv_cache
_PLAN = struct.Struct("13P6q")    # hlwq_kv_plan


def _cache(torch, k_packed, k_norms, v_packed, v_norms, k_window, v_window, requests, n_residual, bits):
    if bits not in (2, 3):
        raise ValueError("bits must be 3 or 2")
    pages, heads, page, _ = _shape(k_packed, 4, "k_packed")
    codes, norms, u8, f16 = (pages, heads, page, 32 * bits), (pages, heads, page), torch.uint8, torch.float16
    kw = vw = ring = 0
    if k_window is not None or v_window is not None or n_residual:
        ring = _shape(k_window, 4, "k_window")[2]
        window, bf16 = (requests, heads, ring, KV_DIM), torch.bfloat16
        kw, vw = _at(k_window, bf16, window, "k_window"), _at(v_window, bf16, window, "v_window")
    return _CACHE.pack(_at(k_packed, u8, codes, "k_packed"), _at(k_norms, f16, norms, "k_norms"), kw,
                       _at(v_packed, u8, codes, "v_packed"), _at(v_norms, f16, norms, "v_norms"), vw, pages, requests,
                       heads, page, n_residual, ring, KV_DIM, bits), heads


def hlwq_kv_page_plan(tokens, n_new, free_pages, n_free, block_table, rows: int, page_size: int = 64,
                      n_residual: int = 128, reset=None, stream=None) -> KvPagePlan:
    """Plan one step of a batch: tokens, n_new int32 [requests] (held and new tokens), free_pages int32 [n_pages] (the
    stack of free page ids, n_free int32 [1] of them), block_table int32 [requests, max_pages]; rows: rows of the
    step's tensors, at least the sum of n_new (rows past it are padding); reset uint8 [requests]: nonzero where the
    slot's request has ended, whose pages go back first.  free_pages and block_table are updated in place."""
    torch = _torch()
    i32 = torch.int32
    n, = _shape(tokens, 1, "tokens")
    pages, = _shape(free_pages, 1, "free_pages")
    width = _shape(block_table, 2, "block_table")[1]
    if rows < 0:
        raise ValueError("rows must not be negative")
    read = (_at(tokens, i32, (n,), "tokens"), _at(n_new, i32, (n,), "n_new"),
            0 if reset is None else _at(reset, torch.uint8, (n,), "reset"), _at(n_free, i32, (1,), "n_free"),
            _at(free_pages, i32, (pages,), "free_pages"), _at(block_table, i32, (n, width), "block_table"))
    out = _empty(2 * n + 3 + 3 * rows, i32, tokens.device, stream)
    plan = KvPagePlan(*out.split_with_sizes((n + 1, n, rows, rows, rows, 1, 1)))
    lens = out.data_ptr() + 4 * (n + 1)
    maps, end = lens + 4 * n, lens + 4 * (n + 3 * rows)
    args = _PLAN.pack(*read, lens - 4 * (n + 1), lens, maps, maps + 4 * rows, maps + 8 * rows, end, end + 4, n, rows, width,
                      pages, page_size, n_residual)
    st = load_library().hlwq_kv_page_plan(args, _stream(stream, (tokens, n_new, free_pages, n_free, block_table, reset)))
    if st:
        _check("hlwq_kv_page_plan", st)
    return plan


def hlwq_kv_paged_append(k_new, v_new, cu_new, lens, row_request, slots, k_packed, k_norms, v_packed, v_norms,
                         k_window, v_window, n_residual: int = 128, bits: int = 3, stream=None):
    """Put a step's keys and values, bf16 [rows, kv_heads, 256] each, into a paged cache: packed uint8
    [n_pages, kv_heads, page_size, 32 * bits], norms fp16 [n_pages, kv_heads, page_size], windows bf16
    [requests, kv_heads, ring, 256] (None when n_residual = 0); cu_new, lens, row_request, slots from the plan."""
    torch = _torch()
    i32, bf16 = torch.int32, torch.bfloat16
    n, = _shape(lens, 1, "lens")
    cache, heads = _cache(torch, k_packed, k_norms, v_packed, v_norms, k_window, v_window, n, n_residual, bits)
    rows = _shape(k_new, 3, "k_new")[0]
    k, ks = _rows(k_new, rows, heads, bf16, "k_new")
    v, vs = _rows(v_new, rows, heads, bf16, "v_new")
    st = load_library().hlwq_kv_paged_append(
        cache, k, ks, v, vs, _at(cu_new, i32, (n + 1,), "cu_new"), _at(lens, i32, (n,), "lens"),
        _at(row_request, i32, (rows,), "row_request"), _at(slots, i32, (rows,), "slots"), rows,
        _stream(stream, (k_new, v_new, cu_new, lens, row_request, slots, k_packed, k_norms, v_packed, v_norms, k_window,
                         v_window)))
    if st:
        _check("hlwq_kv_paged_append", st)


def _heads(q_heads, kv_heads):
    if q_heads and (not kv_heads or q_heads % kv_heads):
        raise ValueError(f"{q_heads} query heads do not divide over {kv_heads} KV heads")


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
    uint8, hlwq_kv_paged_attention_workspace bytes (20 MB for a few single tokens, 135 MB more once there are chunks);
    allocated for the call by default."""
    torch = _torch()
    i32, bf16 = torch.int32, torch.bfloat16
    n, = _shape(lens, 1, "lens")
    cache, heads = _cache(torch, k_packed, k_norms, v_packed, v_norms, k_window, v_window, n, n_residual, bits)
    rows, q_heads, _ = _shape(q, 3, "q")
    _heads(q_heads, heads)
    width = _shape(block_table, 2, "block_table")[1]
    qp, qs = _rows(q, rows, q_heads, bf16, "q")
    k, ks = _rows(k_new, rows, heads, bf16, "k_new")
    v, vs = _rows(v_new, rows, heads, bf16, "v_new")
    cu, le, table = (_at(cu_new, i32, (n + 1,), "cu_new"), _at(lens, i32, (n,), "lens"),
                     _at(block_table, i32, (n, width), "block_table"))
    if out is None:
        out = _empty((rows, q_heads, KV_DIM), bf16, q.device, stream)
    to = _at(out, bf16, (rows, q_heads, KV_DIM), "out")
    lib = load_library()
    if workspace is None:
        workspace = _empty(lib.hlwq_kv_paged_attention_workspace(n, rows, q_heads, heads), torch.uint8, q.device, stream)
    size, = _shape(workspace, 1, "workspace")
    st = lib.hlwq_kv_paged_attention(
        cache, qp, qs, q_heads, k, ks, v, vs, cu, le, table, width, rows, 0.0625 if scale is None else scale, to,
        _at(workspace, torch.uint8, (size,), "workspace"), size,
        _stream(stream, (q, k_new, v_new, cu_new, lens, block_table, k_packed, k_norms, v_packed, v_norms, k_window,
                         v_window, out, workspace)))
    if st:
        _check("hlwq_kv_paged_attention", st)
    return out


def hlwq_prompt_attention(q, k, v, cu_seqlens, scale: float | None = None, out=None, stream=None):
    """Causal attention over whole prompts packed one after the other: q bf16 [rows, q_heads, 256], k and v bf16
    [rows, kv_heads, 256], cu_seqlens int32 [sequences + 1]; scale 1 / 16 by default.  Returns bf16
    [rows, q_heads, 256]; rows past cu_seqlens[-1] are left as they were (undefined in a new `out`)."""
    torch = _torch()
    i32, bf16 = torch.int32, torch.bfloat16
    rows, q_heads, _ = _shape(q, 3, "q")
    heads = _shape(k, 3, "k")[1]
    _heads(q_heads, heads)
    qp, qs = _rows(q, rows, q_heads, bf16, "q")
    kp, ks = _rows(k, rows, heads, bf16, "k")
    vp, vs = _rows(v, rows, heads, bf16, "v")
    ends, = _shape(cu_seqlens, 1, "cu_seqlens")
    if ends < 1:
        raise ValueError("cu_seqlens must have at least one entry")
    cu = _at(cu_seqlens, i32, (ends,), "cu_seqlens")
    if out is None:
        out = _empty((rows, q_heads, KV_DIM), bf16, q.device, stream)
    st = load_library().hlwq_prompt_attention(
        qp, qs, kp, ks, vp, vs, cu, ends - 1, rows, q_heads, heads, KV_DIM, 0.0625 if scale is None else scale,
        _at(out, bf16, (rows, q_heads, KV_DIM), "out"), _stream(stream, (q, k, v, cu_seqlens, out)))
    if st:
        _check("hlwq_prompt_attention", st)
    return out
