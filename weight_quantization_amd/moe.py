"""ctypes binding of libhlwq's mixture-of-experts layer (declared in include/hlwq_moe.h).

A layer of a few tokens from the codes of its banks, as ``hlwq_quantize`` makes them:

    gate_up = hlwq_quantize(w_gate_up)  # [experts, 2 * inner, hidden]: packed, norms
    down = hlwq_quantize(w_down)        # [experts, hidden, inner]
    y = hlwq_moe_layer(x, router, *gate_up, *down, top_k=8).out

As in ``paged``, every function checks its tensors, passes pointers, sizes and the current stream to the C function of
the same name and raises on a status.
"""
from __future__ import annotations

import ctypes
import struct
from typing import TYPE_CHECKING, NamedTuple

from . import binding
from .binding import BLOCK, _check, _i64, _int, _torch, _vp, load_library
from .paged import _at, _empty, _fail, _shape, _stream

if TYPE_CHECKING:
    import torch


binding._SIGNATURES.update({
    "hlwq_moe_experts": (_int, [_vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "hlwq_moe_layer": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _int, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "hlwq_moe_workspace": (ctypes.c_size_t, [_i64, _i64, _i64, _i64, _i64]),
})

_BANKS = struct.Struct("4P3q2i")  # hlwq_moe_banks
_ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}


class MoeOutput(NamedTuple):
    out: torch.Tensor      # bf16 [tokens, hidden]
    experts: torch.Tensor  # int32 [tokens, top_k]
    weights: torch.Tensor  # fp32 [tokens, top_k]


def _banks(torch, gate_up_packed, gate_up_norms, down_packed, down_norms, hidden, bits, activation):
    if bits not in (5, 3):
        raise ValueError("bits must be 5 or 3")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}")
    experts, both, _, _ = _shape(gate_up_packed, 4, "gate_up_packed")
    if both % 2:
        raise ValueError(f"gate_up_packed must have as many rows of gate as of up, got {both}")
    inner = both // 2
    up, down = (experts, both, -(-hidden // BLOCK)), (experts, hidden, -(-inner // BLOCK))
    u8, f16 = torch.uint8, torch.float16
    return _BANKS.pack(_at(gate_up_packed, u8, (*up, 16 * bits), "gate_up_packed"), _at(gate_up_norms, f16, up, "gate_up_norms"),
                       _at(down_packed, u8, (*down, 16 * bits), "down_packed"), _at(down_norms, f16, down, "down_norms"),
                       experts, hidden, inner, bits, _ACTIVATIONS[activation]), experts, inner


def _x(t, bf16):
    """Tokens [tokens, hidden] in bf16, whole rows at any stride (the C function takes strides up to 2^20).  Returns the
    address and the stride."""
    tokens, hidden = _shape(t, 2, "x")
    if t.dtype is not bf16 or not t.is_cuda:
        _fail(t, bf16, "x")
    row, one = t.stride()
    if tokens <= 1:
        row = hidden  # there is no next row
    if t.numel() and ((one != 1 and hidden > 1) or row < hidden):
        raise ValueError(f"x must hold each row's values side by side; its strides are {t.stride()}")
    return t.data_ptr(), row, tokens, hidden


def _buffers(torch, lib, out, workspace, experts, hidden, inner, tokens, top_k, device, stream):
    if out is None:
        out = _empty((tokens, hidden), torch.bfloat16, device, stream)
    to = _at(out, torch.bfloat16, (tokens, hidden), "out")
    if workspace is None:
        workspace = _empty(lib.hlwq_moe_workspace(experts, hidden, inner, tokens, top_k), torch.uint8, device, stream)
    size, = _shape(workspace, 1, "workspace")
    return out, to, workspace, _at(workspace, torch.uint8, (size,), "workspace"), size


def hlwq_moe_workspace(experts: int, hidden: int, inner: int, tokens: int, top_k: int) -> int:
    """Bytes of workspace that hlwq_moe_experts and hlwq_moe_layer need for these sizes."""
    return int(load_library().hlwq_moe_workspace(experts, hidden, inner, tokens, top_k))


def hlwq_moe_experts(x, experts, weights, gate_up_packed, gate_up_norms, down_packed, down_norms, bits: int = 5,
                     activation: str = "silu", out=None, workspace=None, stream=None):
    """The weighted sum of the experts' outputs for tokens whose routing is known: x bf16 [tokens, hidden] (rows at most
    2^20 elements apart), experts int32 and weights fp32 [tokens, top_k], the banks' codes as hlwq_quantize returns them
    for [experts, 2 * inner, hidden] (gate rows, then up rows) and [experts, hidden, inner]; activation "silu" or
    "gelu_tanh".  Returns bf16 [tokens, hidden].  workspace: uint8, hlwq_moe_workspace bytes; allocated for the call by
    default."""
    torch = _torch()
    xp, xs, tokens, hidden = _x(x, torch.bfloat16)
    banks, n, inner = _banks(torch, gate_up_packed, gate_up_norms, down_packed, down_norms, hidden, bits, activation)
    k = _shape(experts, 2, "experts")[1]
    ids, w = _at(experts, torch.int32, (tokens, k), "experts"), _at(weights, torch.float32, (tokens, k), "weights")
    lib = load_library()
    out, to, workspace, ws, size = _buffers(torch, lib, out, workspace, n, hidden, inner, tokens, k, x.device, stream)
    st = lib.hlwq_moe_experts(banks, xp, xs, tokens, k, ids, w, to, ws, size,
                              _stream(stream, (x, experts, weights, gate_up_packed, gate_up_norms, down_packed, down_norms, out,
                                               workspace)))
    if st:
        _check("hlwq_moe_experts", st)
    return out


def hlwq_moe_layer(x, router, gate_up_packed, gate_up_norms, down_packed, down_norms, top_k: int, bits: int = 5,
                   activation: str = "silu", renormalize: bool = True, out=None, workspace=None, stream=None) -> MoeOutput:
    """A mixture-of-experts layer: as hlwq_moe_experts, the experts of each token being the top_k of router (bf16
    [experts, hidden]) times x, ties to the lower index, and their weights the softmax over all experts, or with
    renormalize over the chosen ones.  Returns the output, the experts and their weights."""
    torch = _torch()
    xp, xs, tokens, hidden = _x(x, torch.bfloat16)
    banks, n, inner = _banks(torch, gate_up_packed, gate_up_norms, down_packed, down_norms, hidden, bits, activation)
    if not 0 <= top_k <= n:
        raise ValueError(f"top_k must be between 0 and the {n} experts")
    r = _at(router, torch.bfloat16, (n, hidden), "router")
    both = _empty((2, tokens, top_k), torch.int32, x.device, stream)
    ids, weights = both[0], both[1].view(torch.float32)
    lib = load_library()
    out, to, workspace, ws, size = _buffers(torch, lib, out, workspace, n, hidden, inner, tokens, top_k, x.device, stream)
    at = both.data_ptr()
    st = lib.hlwq_moe_layer(banks, xp, xs, tokens, r, top_k, bool(renormalize), at, at + 4 * tokens * top_k, to, ws, size,
                            _stream(stream, (x, router, gate_up_packed, gate_up_norms, down_packed, down_norms, out, workspace)))
    if st:
        _check("hlwq_moe_layer", st)
    return MoeOutput(out, ids, weights)
