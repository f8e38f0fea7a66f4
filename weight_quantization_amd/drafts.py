"""ctypes binding of libhlwq's operators for trees of drafted tokens (declared in include/hlwq_drafts.h).

Attention of the trees over a paged cache, and which of their tokens stand against the target's probabilities.  A step
drafts a tree of rows for each request, whose first row is its last token:

    out = hlwq_kv_tree_attention(q, k, v, parents, cu_rows, lens, block_table, *cache)  # each layer
    v = hlwq_verify_drafts(tokens, parents, cu_rows, target, uniforms, next_uniforms, draft)

As in ``paged``, every function checks its tensors, passes pointers, sizes and the current stream to the C function of
the same name and raises on a status.
"""
from __future__ import annotations

import ctypes
import struct
from typing import TYPE_CHECKING, NamedTuple

from . import binding
from .binding import KV_DIM, _check, _i64, _int, _torch, _vp, load_library
from .paged import _at, _cache, _empty, _heads, _rows, _shape, _stream

if TYPE_CHECKING:
    import torch


binding._SIGNATURES.update({
    "hlwq_kv_tree_attention": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp,
                                      _i64, _i64, ctypes.c_float, _vp, _vp, ctypes.c_size_t, _vp]),
    "hlwq_kv_tree_attention_workspace": (ctypes.c_size_t, [_i64, _i64, _i64, _i64]),
    "hlwq_verify_drafts": (_int, [_vp, _vp]),
})

_DRAFTS = struct.Struct("10P5qi4x")  # hlwq_drafts


class VerifiedDrafts(NamedTuple):
    """What hlwq_verify_drafts writes, int32 on the device."""
    n_kept: torch.Tensor      # [requests] rows kept, the root among them
    next_token: torch.Tensor  # [requests] the token that follows them
    kept: torch.Tensor        # [rows] rows kept, a request's from its first row's place on; -1 elsewhere


def hlwq_kv_tree_attention_workspace(requests: int, rows: int, q_heads: int, kv_heads: int) -> int:
    """Bytes of workspace that hlwq_kv_tree_attention needs for these sizes."""
    return int(load_library().hlwq_kv_tree_attention_workspace(requests, rows, q_heads, kv_heads))


def hlwq_kv_tree_attention(q, k_new, v_new, parents, cu_rows, lens, block_table, k_packed, k_norms, v_packed, v_norms,
                           k_window, v_window, n_residual: int = 128, bits: int = 3, scale: float | None = None,
                           out=None, workspace=None, stream=None):
    """Attention of trees of rows over pages, window and each row's own ancestors: as hlwq_kv_paged_attention, with
    parents int32 [rows] the index, within its request, of the row that each row follows (less than its own), or -1
    where it follows the cached tokens; cu_rows int32 [requests + 1] the trees' rows, lens int32 [requests] tokens held
    plus rows.  Returns bf16 [rows, q_heads, 256]; rows past cu_rows[requests] are left as they were (undefined in a
    new `out`).  workspace: uint8, hlwq_kv_tree_attention_workspace bytes; allocated for the call by default."""
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
    tree, cu, le, table = (_at(parents, i32, (rows,), "parents"), _at(cu_rows, i32, (n + 1,), "cu_rows"),
                           _at(lens, i32, (n,), "lens"), _at(block_table, i32, (n, width), "block_table"))
    if out is None:
        out = _empty((rows, q_heads, KV_DIM), bf16, q.device, stream)
    to = _at(out, bf16, (rows, q_heads, KV_DIM), "out")
    lib = load_library()
    if workspace is None:
        workspace = _empty(lib.hlwq_kv_tree_attention_workspace(n, rows, q_heads, heads), torch.uint8, q.device, stream)
    size, = _shape(workspace, 1, "workspace")
    st = lib.hlwq_kv_tree_attention(
        cache, qp, qs, q_heads, k, ks, v, vs, tree, cu, le, table, width, rows, 0.0625 if scale is None else scale, to,
        _at(workspace, torch.uint8, (size,), "workspace"), size,
        _stream(stream, (q, k_new, v_new, parents, cu_rows, lens, block_table, k_packed, k_norms, v_packed, v_norms, k_window,
                         v_window, out, workspace)))
    if st:
        _check("hlwq_kv_tree_attention", st)
    return out


def _probabilities(t, rows, vocab, dtype, name):
    """Rows of probabilities [rows, vocab] of this type, any row stride.  Returns the address and the stride."""
    torch = _torch()
    shape = _shape(t, 2, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be in device memory")
    if tuple(shape) != (rows, vocab):
        raise ValueError(f"{name} must have shape {[rows, vocab]}, got {list(shape)}")
    row, one = t.stride()
    if rows <= 1:
        row = vocab  # there is no next row
    if t.numel() and ((one != 1 and vocab > 1) or row < vocab):
        raise ValueError(f"{name} must hold each row's values side by side; its strides are {t.stride()}")
    return t.data_ptr(), row


def hlwq_verify_drafts(tokens, parents, cu_rows, target, uniforms, next_uniforms, draft=None, stream=None) -> VerifiedDrafts:
    """Which drafted tokens stand, and the token that follows them, distributed as the target's own samples: tokens,
    parents int32 [rows] and cu_rows int32 [requests + 1] the trees (as in hlwq_kv_tree_attention; a request's row 0 is
    its last token), target [rows, vocab] the target's probabilities of the token after each row, draft [rows, vocab]
    what the tokens of a row's children were drawn from (None: they were not drawn at random), both fp32, bf16 or fp16;
    uniforms fp32 [rows] decide on the rows' tokens, next_uniforms fp32 [requests] on the tokens that follow."""
    torch = _torch()
    i32, f32 = torch.int32, torch.float32
    rows, vocab = _shape(target, 2, "target")
    n, = _shape(next_uniforms, 1, "next_uniforms")
    kind = {f32: 0, torch.bfloat16: 1, torch.float16: 2}.get(target.dtype)
    if kind is None:
        raise TypeError(f"target must be fp32, bf16 or fp16, got {target.dtype}")
    if vocab < 1:
        raise ValueError("target must have at least one token to a row")
    p, ps = _probabilities(target, rows, vocab, target.dtype, "target")
    q, qs = (0, vocab) if draft is None else _probabilities(draft, rows, vocab, target.dtype, "draft")
    read = (_at(tokens, i32, (rows,), "tokens"), _at(parents, i32, (rows,), "parents"), _at(cu_rows, i32, (n + 1,), "cu_rows"),
            p, q, _at(uniforms, f32, (rows,), "uniforms"), _at(next_uniforms, f32, (n,), "next_uniforms"))
    out = _empty(2 * n + rows, i32, target.device, stream)
    result = VerifiedDrafts(*out.split_with_sizes((n, n, rows)))
    at = out.data_ptr()
    args = _DRAFTS.pack(*read, at, at + 4 * n, at + 8 * n, n, rows, vocab, ps, qs, kind)
    st = load_library().hlwq_verify_drafts(args, _stream(stream, (tokens, parents, cu_rows, target, uniforms, next_uniforms,
                                                                   draft)))
    if st:
        _check("hlwq_verify_drafts", st)
    return result
