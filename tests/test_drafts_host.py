"""Host-side checks of the operators of drafted tokens and of the experts' layer (CPU only, no kernel is launched)."""
import ctypes
import os
import re

import pytest

import weight_quantization_amd as wq
from test_paged_host import (A, EALIGN, EBITS, EBLOCK, ELIMIT, ENULL, EOVERLAP, ESHAPE, OK, at, cache,  # noqa: F401
                             lib)

INCLUDE = os.path.dirname(wq.binding.HEADER_PATH)


@pytest.mark.parametrize("header,names", [
    ("hlwq_drafts.h", ["hlwq_kv_tree_attention", "hlwq_kv_tree_attention_workspace", "hlwq_verify_drafts"]),
    ("hlwq_moe.h", ["hlwq_moe_experts", "hlwq_moe_layer", "hlwq_moe_workspace"])])
def test_exports_every_declared_symbol(lib, header, names):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, header)).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(hlwq_[a-z_0-9]+)\s*\(", text))) == names
    raw = ctypes.CDLL(wq.binding.LIB_PATH)
    for n in names:
        assert hasattr(raw, n) and n in wq.binding._SIGNATURES and n in dir(wq)


# ---------------------------------------------------------------------------
# attention of trees
# ---------------------------------------------------------------------------

def tree(lib, c, q=at(12), qs=6144, hq=24, k=at(6), ks=1024, v=at(7), vs=1024, parents=at(16), cu=at(8), lens=at(9),
         table=at(13), width=9, rows=5, scale=0.0625, out=at(14), ws=at(15), bytes_=2 ** 34):
    return lib.hlwq_kv_tree_attention(ctypes.byref(c), q, qs, hq, k, ks, v, vs, parents, cu, lens, table, width, rows, scale,
                                      out, ws, bytes_, None)


def test_tree_argument_errors(lib):
    c = cache()
    for name in ("q", "k", "v", "cu", "lens", "table", "out", "ws", "parents"):
        assert tree(lib, c, **{name: None}) == ENULL, name
    for name, value in (("q", at(12) + 8), ("k", at(6) + 2), ("parents", at(16) + 2), ("cu", at(8) + 1), ("lens", at(9) + 2),
                        ("table", at(13) + 3), ("out", at(14) + 8), ("ws", at(15) + 4)):
        assert tree(lib, c, **{name: value}) == EALIGN, name
    assert tree(lib, c, qs=6136) == ESHAPE and tree(lib, c, ks=1016) == ESHAPE and tree(lib, c, hq=23) == ESHAPE
    assert tree(lib, c, rows=-1) == ESHAPE and tree(lib, c, width=-1) == ESHAPE and tree(lib, c, scale=float("inf")) == ESHAPE
    assert tree(lib, c, bytes_=100) == ESHAPE
    assert tree(lib, c, width=2 ** 20 + 1) == ELIMIT and tree(lib, c, qs=2 ** 22 + 8) == ELIMIT
    assert tree(lib, c, rows=2 ** 28) == ELIMIT
    assert tree(lib, cache(bits=5)) == EBITS and tree(lib, cache(head_dim=128)) == EBLOCK
    for name in ("q", "k", "parents", "cu", "lens", "table", "ws"):
        assert tree(lib, c, out={"q": at(12), "k": at(6), "parents": at(16), "cu": at(8), "lens": at(9), "table": at(13),
                                 "ws": at(15)}[name]) == EOVERLAP, name
    assert tree(lib, c, out=at(2)) == EOVERLAP
    assert tree(lib, c, rows=0, q=None, parents=None, out=None, ws=None) == OK
    assert lib.hlwq_kv_tree_attention(None, *[None] * 0, at(12), 6144, 24, at(6), 1024, at(7), 1024, at(16), at(8), at(9), at(13), 9,
                                      5, 0.0625, at(14), at(15), 2 ** 34, None) == ENULL


def test_tree_workspace():
    w = wq.hlwq_kv_tree_attention_workspace
    tile = 2 * 16 * 258 * 4
    assert w(64, 64, 24, 4) == (512 + (64 * 6 // 16 + 64) * 4) * tile
    # many rows to a request: room for tiles of 64 too, whichever is more
    assert w(1, 4096, 24, 4) == (256 + (4096 * 6 // 64 + 1) * 4) * 4 * tile + 4096 * 24 * 516
    assert w(1, 31, 24, 4) == (512 + 12 * 4) * tile  # 186 rows of a KV head
    assert w(4, 31, 24, 4) == (512 + (31 * 6 // 16 + 4) * 4) * tile
    assert w(1, 1, 24, 4) == 512 * tile  # four tiles' workgroups have places among the 512
    for bad in ((0, 5, 24, 4), (-1, 5, 24, 4), (1, 0, 24, 4), (1, 5, 23, 4), (1, 5, 24, 0), (2 ** 20 + 1, 5, 24, 4),
                (1, 2 ** 27, 24, 4), (2 ** 20, 2 ** 20, 1, 1)):
        assert w(*bad) == 0, bad


# ---------------------------------------------------------------------------
# verification
# ---------------------------------------------------------------------------

class Drafts(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("tokens", "parents", "cu_rows", "target", "draft", "uniforms", "next_uniforms",
                                               "n_kept", "next_token", "kept")]
    _fields_ += [(n, ctypes.c_int64) for n in ("requests", "rows", "vocab", "target_stride", "draft_stride")]
    _fields_ += [("dtype", ctypes.c_int)]


def verify(lib, **kw):
    d = dict(tokens=at(0), parents=at(1), cu_rows=at(2), target=at(3), draft=at(4), uniforms=at(5), next_uniforms=at(6),
             n_kept=at(7), next_token=at(8), kept=at(9), requests=3, rows=7, vocab=100, target_stride=100, draft_stride=100, dtype=0)
    d.update(kw)
    return lib.hlwq_verify_drafts(ctypes.byref(Drafts(**d)), None)


def test_verify_argument_errors(lib):
    assert lib.hlwq_verify_drafts(None, None) == ENULL
    for name in ("tokens", "parents", "cu_rows", "target", "uniforms", "next_uniforms", "n_kept", "next_token", "kept"):
        assert verify(lib, **{name: None}) == ENULL, name
        assert verify(lib, **{name: at(20) + 2}) == EALIGN, name
    assert verify(lib, draft=at(4) + 1) == EALIGN and verify(lib, target=at(3) + 1, dtype=1) == EALIGN
    for kw in (dict(dtype=3), dict(dtype=-1), dict(requests=-1), dict(rows=-1), dict(vocab=0), dict(vocab=-5),
               dict(target_stride=99), dict(draft_stride=99)):
        assert verify(lib, **kw) == ESHAPE, kw
    for kw in (dict(requests=2 ** 20 + 1), dict(rows=2 ** 31), dict(vocab=2 ** 24 + 1, target_stride=2 ** 25, draft_stride=2 ** 25),
               dict(target_stride=2 ** 40 + 1), dict(draft_stride=2 ** 40 + 1)):
        assert verify(lib, **kw) == ELIMIT, kw
    for out in ("n_kept", "next_token", "kept"):
        for other in range(10):
            if at(other) != {"n_kept": at(7), "next_token": at(8), "kept": at(9)}[out]:
                assert verify(lib, **{out: at(other)}) == EOVERLAP, (out, other)
    # past the buffers by the stride
    assert verify(lib, target_stride=2 ** 34, vocab=100, draft=at(4), n_kept=at(3) + 6 * 2 ** 36) == EOVERLAP
    assert verify(lib, requests=0, tokens=None, target=None, kept=None, n_kept=None) == OK


# ---------------------------------------------------------------------------
# experts' layer
# ---------------------------------------------------------------------------

class Banks(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("gate_up_packed", "gate_up_norms", "down_packed", "down_norms")]
    _fields_ += [(n, ctypes.c_int64) for n in ("experts", "hidden", "inner")]
    _fields_ += [("bits", ctypes.c_int), ("activation", ctypes.c_int)]


def banks(**kw):
    d = dict(gate_up_packed=at(0), gate_up_norms=at(1), down_packed=at(2), down_norms=at(3), experts=8, hidden=256, inner=130, bits=5,
             activation=0)
    d.update(kw)
    return Banks(**d)


def layer(lib, b, x=at(4), xs=256, tokens=3, router=at(5), k=2, ids=at(6), w=at(7), out=at(8), ws=at(9), bytes_=2 ** 34):
    return lib.hlwq_moe_layer(ctypes.byref(b), x, xs, tokens, router, k, 1, ids, w, out, ws, bytes_, None)


def given(lib, b, x=at(4), xs=256, tokens=3, k=2, ids=at(6), w=at(7), out=at(8), ws=at(9), bytes_=2 ** 34):
    return lib.hlwq_moe_experts(ctypes.byref(b), x, xs, tokens, k, ids, w, out, ws, bytes_, None)


def test_moe_argument_errors(lib):
    for call in (layer, given):
        for name in ("x", "ids", "w", "out", "ws"):
            assert call(lib, banks(), **{name: None}) == ENULL, name
        for name in ("gate_up_packed", "gate_up_norms", "down_packed", "down_norms"):
            assert call(lib, banks(**{name: None})) == ENULL, name
            assert call(lib, banks(**{name: at(20) + 1})) == EALIGN, name
            assert call(lib, banks(), out=getattr(banks(), name)) == EOVERLAP, name
        for name, by in (("x", 1), ("ids", 2), ("w", 1), ("out", 1), ("ws", 8)):
            assert call(lib, banks(), **{name: at(20) + by}) == EALIGN, name
        assert call(lib, banks(bits=4)) == EBITS and call(lib, banks(bits=2)) == EBITS
        for kw in (dict(activation=2), dict(activation=-1), dict(experts=-1), dict(hidden=-1), dict(inner=-1)):
            assert call(lib, banks(**kw)) == ESHAPE, kw
        assert call(lib, banks(), tokens=-1) == ESHAPE and call(lib, banks(), k=-1) == ESHAPE
        assert call(lib, banks(), xs=255) == ESHAPE and call(lib, banks(), bytes_=100) == ESHAPE
        for kw in (dict(experts=1025), dict(hidden=2 ** 20 + 1), dict(inner=2 ** 20 + 1), dict(hidden=2 ** 17, inner=2 ** 17)):
            assert call(lib, banks(**kw), xs=2 ** 20) == ELIMIT, kw
        assert call(lib, banks(), tokens=2 ** 24 + 1) == ELIMIT and call(lib, banks(), xs=2 ** 20 + 1) == ELIMIT
        assert call(lib, banks(), k=33) == ELIMIT
        for name in ("x", "ids", "w", "ws"):
            assert call(lib, banks(), out={"x": at(4), "ids": at(6), "w": at(7), "ws": at(9)}[name]) == EOVERLAP, name
        assert call(lib, banks(), tokens=0, x=None, ids=None, w=None, out=None, ws=None) == OK
    assert layer(lib, banks(), router=None) == ENULL and layer(lib, banks(), router=at(5) + 1) == EALIGN
    assert layer(lib, banks(), k=9) == ESHAPE
    assert layer(lib, banks(), ids=at(5)) == EOVERLAP and layer(lib, banks(), w=at(4)) == EOVERLAP
    assert layer(lib, banks(), w=at(6)) == EOVERLAP
    assert lib.hlwq_moe_experts(None, at(4), 256, 3, 2, at(6), at(7), at(8), at(9), 2 ** 34, None) == ENULL


def test_moe_workspace():
    w = wq.hlwq_moe_workspace
    assert w(256, 2048, 512, 64, 8) > 512 * 2048 * 4
    # tokens are taken 4096 / top_k at a time
    assert w(256, 2048, 512, 512, 8) == w(256, 2048, 512, 100000, 8)
    for bad in ((1025, 2048, 512, 1, 8), (256, 2 ** 20 + 1, 512, 1, 8), (-1, 2048, 512, 1, 8), (256, 2048, 512, 0, 8),
                (256, 2048, 512, 1, 33), (256, 2048, 512, 2 ** 24 + 1, 8), (256, 0, 512, 1, 8)):
        assert w(*bad) == 0, bad


def test_python_refusals_without_a_device():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        wq.hlwq_moe_layer(x, x, x, x, x, x, top_k=1)
    with pytest.raises(TypeError):
        wq.hlwq_moe_layer(None, x, x, x, x, x, top_k=1)
    with pytest.raises(ValueError):
        wq.hlwq_verify_drafts(x, x, x, torch.zeros(2, 9), x, torch.zeros(1))
    with pytest.raises(TypeError):
        wq.hlwq_kv_tree_attention(None, None, None, None, None, None, None, None, None, None, None, None, None)


def test_routing_of_rows_of_nothing_checks_what_it_writes(lib):
    b = banks(hidden=0)
    assert given(lib, b, xs=0, x=None, ids=None, w=None, out=None, ws=None) == OK
    assert layer(lib, b, xs=0, k=0, x=None, ids=None, w=None, out=None, ws=None) == OK
    assert layer(lib, b, xs=0, tokens=0, x=None, ids=None, w=None, out=None, ws=None) == OK
    none = dict(xs=0, x=None, out=None, ws=None)
    assert layer(lib, b, ids=None, **none) == ENULL and layer(lib, b, w=None, **none) == ENULL
    assert layer(lib, b, ids=at(6) + 1, **none) == EALIGN and layer(lib, b, w=at(7) + 2, **none) == EALIGN
    assert layer(lib, b, w=at(6) + 20, **none) == EOVERLAP and layer(lib, b, k=9, **none) == ESHAPE
