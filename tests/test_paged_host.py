"""Host-side checks of the serving operators (CPU only, no kernel is launched)."""
import ctypes
import math
import os
import re

import pytest

import weight_quantization_amd as wq
from weight_quantization_amd import paged

OK, ENULL, ESHAPE, EBITS, EBLOCK, EDEV, EALIGN, ELIMIT, EOVERLAP = 0, -1, -2, -3, -4, -5, -6, -7, -8
HEADER = os.path.join(os.path.dirname(wq.binding.HEADER_PATH), "hlwq_attention.h")


class KvStore(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("packed", "norms", "window")]


class KvCache(ctypes.Structure):
    _fields_ = [("k", KvStore), ("v", KvStore)]
    _fields_ += [(n, ctypes.c_int64) for n in ("n_pages", "requests", "kv_heads", "page_size", "n_residual", "ring")]
    _fields_ += [("head_dim", ctypes.c_int), ("bits", ctypes.c_int)]


class KvPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("tokens", "n_new", "reset", "n_free", "free_pages", "block_table", "cu_new",
                                               "lens", "row_request", "positions", "slots", "n_free_after", "status")]
    _fields_ += [(n, ctypes.c_int64) for n in ("requests", "rows", "max_pages", "n_pages", "page_size", "n_residual")]


A = 1 << 32  # aligned addresses far apart, never dereferenced
STEP = 1 << 36


def at(k):
    return A + k * STEP


@pytest.fixture(scope="module")
def lib():
    return wq.load_library()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(hlwq_[a-z_0-9]+)\s*\(", text)))
    assert names == ["hlwq_kv_page_plan", "hlwq_kv_paged_append", "hlwq_kv_paged_attention",
                     "hlwq_kv_paged_attention_workspace", "hlwq_prompt_attention"]
    raw = ctypes.CDLL(wq.binding.LIB_PATH)
    for n in names:
        assert hasattr(raw, n), n
        assert n in wq.binding._SIGNATURES


def cache(**kw):
    d = dict(n_pages=8, requests=2, kv_heads=4, page_size=64, n_residual=128, ring=128, head_dim=256, bits=3)
    d.update({k: v for k, v in kw.items() if k not in ("k", "v")})
    k = KvStore(*kw.get("k", (at(0), at(1), at(2))))
    v = KvStore(*kw.get("v", (at(3), at(4), at(5))))
    return KvCache(k, v, d["n_pages"], d["requests"], d["kv_heads"], d["page_size"], d["n_residual"], d["ring"],
                         d["head_dim"], d["bits"])


CACHE_FAULTS = [
    (dict(head_dim=128), EBLOCK), (dict(bits=5), EBITS), (dict(bits=4), EBITS), (dict(n_pages=-1), ESHAPE),
    (dict(requests=-1), ESHAPE), (dict(kv_heads=-1), ESHAPE), (dict(n_residual=-1), ESHAPE), (dict(ring=127), ESHAPE),
    (dict(page_size=8), ESHAPE), (dict(page_size=48), ESHAPE), (dict(page_size=512), ESHAPE), (dict(page_size=0), ESHAPE),
    (dict(n_pages=2 ** 31 // 64), ELIMIT), (dict(requests=2 ** 20 + 1), ELIMIT), (dict(kv_heads=2 ** 12 + 1), ELIMIT),
    (dict(ring=2 ** 31), ELIMIT), (dict(k=(None, at(1), at(2))), ENULL), (dict(k=(at(0), None, at(2))), ENULL),
    (dict(v=(at(3), at(4), None)), ENULL), (dict(k=(at(0) + 8, at(1), at(2))), EALIGN),
    (dict(v=(at(3), at(4) + 1, at(5))), EALIGN), (dict(v=(at(3), at(4), at(5) + 2)), EALIGN),
]


@pytest.mark.parametrize("kw,status", CACHE_FAULTS)
def test_cache_faults(lib, kw, status):
    c = cache(**kw)
    assert lib.hlwq_kv_paged_append(ctypes.byref(c), at(6), 1024, at(7), 1024, at(8), at(9), at(10), at(11), 5,
                                    None) == status
    assert attention(lib, c) == status


def append(lib, c, k=at(6), ks=1024, v=at(7), vs=1024, cu=at(8), lens=at(9), req=at(10), slots=at(11), rows=5):
    return lib.hlwq_kv_paged_append(ctypes.byref(c), k, ks, v, vs, cu, lens, req, slots, rows, None)


def attention(lib, c, q=at(12), qs=6144, hq=24, k=at(6), ks=1024, v=at(7), vs=1024, cu=at(8), lens=at(9), table=at(13),
              width=9, rows=5, scale=0.0625, out=at(14), ws=at(15), bytes_=2 ** 34):
    return lib.hlwq_kv_paged_attention(ctypes.byref(c), q, qs, hq, k, ks, v, vs, cu, lens, table, width, rows, scale, out,
                                       ws, bytes_, None)


def test_append_argument_errors(lib):
    c = cache()
    assert append(lib, c, k=None) == ENULL
    assert append(lib, c, v=None) == ENULL
    assert append(lib, c, cu=None) == ENULL
    assert append(lib, c, lens=None) == ENULL
    assert append(lib, c, req=None) == ENULL
    assert append(lib, c, slots=None) == ENULL
    assert append(lib, c, ks=1016) == ESHAPE
    assert append(lib, c, vs=1028) == ESHAPE
    assert append(lib, c, ks=2 ** 22 + 8) == ELIMIT
    assert append(lib, c, rows=-1) == ESHAPE
    assert append(lib, c, rows=2 ** 31) == ELIMIT
    assert append(lib, c, k=at(6) + 8) == EALIGN
    assert append(lib, c, slots=at(11) + 2) == EALIGN
    assert append(lib, c, k=at(0)) == EOVERLAP          # keys in the written pages
    assert append(lib, c, slots=at(5) + 512) == EOVERLAP  # slots in a window
    assert append(lib, cache(v=(at(0), at(4), at(5)))) == EOVERLAP
    assert append(lib, c, rows=0, k=None, v=None, cu=None) == OK
    assert append(lib, cache(requests=0, k=(at(0), at(1), None), v=(at(3), at(4), None))) == OK
    assert lib.hlwq_kv_paged_append(None, at(6), 1024, at(7), 1024, at(8), at(9), at(10), at(11), 5, None) == ENULL


def test_attention_argument_errors(lib):
    c = cache()
    for name in ("q", "k", "v", "cu", "lens", "table", "out", "ws"):
        assert attention(lib, c, **{name: None}) == ENULL, name
    assert attention(lib, c, hq=22) == ESHAPE
    assert attention(lib, c, hq=-4) == ESHAPE
    assert attention(lib, cache(kv_heads=0)) == ESHAPE
    assert attention(lib, c, qs=6136) == ESHAPE
    assert attention(lib, c, qs=6146) == ESHAPE
    assert attention(lib, c, rows=-1) == ESHAPE
    assert attention(lib, c, width=-1) == ESHAPE
    assert attention(lib, c, scale=math.nan) == ESHAPE
    assert attention(lib, c, scale=math.inf) == ESHAPE
    assert attention(lib, c, width=2 ** 20 + 1) == ELIMIT
    assert attention(lib, c, rows=2 ** 31) == ELIMIT
    assert attention(lib, c, hq=2 ** 12 + 4, qs=2 ** 21) == ELIMIT
    assert attention(lib, c, q=at(12) + 2) == EALIGN
    assert attention(lib, c, out=at(14) + 8) == EALIGN
    assert attention(lib, c, ws=at(15) + 8) == EALIGN
    assert attention(lib, c, table=at(13) + 1) == EALIGN
    assert attention(lib, c, out=at(12) + 512) == EOVERLAP
    assert attention(lib, c, ws=at(2)) == EOVERLAP
    need = lib.hlwq_kv_paged_attention_workspace(2, 5, 24, 4)
    assert need > 0
    assert attention(lib, c, bytes_=need - 1) == ESHAPE
    assert attention(lib, c, rows=0, q=None, out=None, ws=None) == OK
    assert attention(lib, c, hq=0, q=None, out=None, ws=None) == OK


def test_workspace_helper():
    w = wq.hlwq_kv_paged_attention_workspace
    assert w(0, 5, 24, 4) == 0 and w(2, 0, 24, 4) == 0 and w(2, 5, 23, 4) == 0 and w(2, 5, 24, 0) == 0
    assert w(-1, 5, 24, 4) == 0 and w(2 ** 21, 5, 24, 4) == 0
    assert w(1, 1, 24, 4) > 0 and w(2 ** 20, 2 ** 31 // 4096 - 1, 4096, 1) > 0 and w(1, 2 ** 31 // 4096, 4096, 1) == 0


def prompt(lib, q=at(0), qs=6144, k=at(1), ks=1024, v=at(2), vs=1024, cu=at(3), n=2, rows=5, hq=24, hk=4, d=256,
           scale=0.0625, out=at(4)):
    return lib.hlwq_prompt_attention(q, qs, k, ks, v, vs, cu, n, rows, hq, hk, d, scale, out, None)


def test_prompt_argument_errors(lib):
    for name in ("q", "k", "v", "cu", "out"):
        assert prompt(lib, **{name: None}) == ENULL, name
    assert prompt(lib, d=128) == EBLOCK
    assert prompt(lib, hq=23) == ESHAPE
    assert prompt(lib, hk=0) == ESHAPE
    assert prompt(lib, n=-1) == ESHAPE
    assert prompt(lib, rows=-1) == ESHAPE
    assert prompt(lib, qs=6140) == ESHAPE
    assert prompt(lib, ks=1020) == ESHAPE
    assert prompt(lib, vs=1000) == ESHAPE
    assert prompt(lib, scale=-math.inf) == ESHAPE
    assert prompt(lib, n=2 ** 20 + 1) == ELIMIT
    assert prompt(lib, rows=2 ** 31) == ELIMIT
    assert prompt(lib, k=at(1) + 2) == EALIGN
    assert prompt(lib, out=at(4) + 2) == EALIGN
    assert prompt(lib, cu=at(3) + 2) == EALIGN
    assert prompt(lib, out=at(0)) == EOVERLAP
    assert prompt(lib, out=at(2) + 1024) == EOVERLAP
    assert prompt(lib, rows=0, q=None, k=None, v=None, cu=None, out=None) == OK
    assert prompt(lib, n=0, q=None, k=None, v=None, cu=None, out=None) == OK


def plan_args(**kw):
    d = {n: at(i) for i, n in enumerate(("tokens", "n_new", "reset", "n_free", "free_pages", "block_table", "cu_new", "lens",
                                         "row_request", "positions", "slots", "n_free_after", "status"))}
    d.update(requests=3, rows=7, max_pages=5, n_pages=11, page_size=64, n_residual=128)
    d.update(kw)
    return KvPlan(**d)


@pytest.mark.parametrize("kw,status", [
    *((({n: None}), ENULL) for n in ("tokens", "n_new", "n_free", "free_pages", "block_table", "cu_new", "lens",
                                     "row_request", "positions", "slots", "n_free_after", "status")),
    *((({n: -1}), ESHAPE) for n in ("requests", "rows", "max_pages", "n_pages", "n_residual")),
    (dict(page_size=100), ESHAPE), (dict(page_size=8), ESHAPE), (dict(page_size=1024), ESHAPE),
    (dict(requests=2 ** 20 + 1), ELIMIT), (dict(max_pages=2 ** 20 + 1), ELIMIT), (dict(rows=2 ** 31), ELIMIT),
    (dict(n_pages=2 ** 31 // 64), ELIMIT), (dict(slots=at(20) + 2), EALIGN), (dict(lens=at(0)), EOVERLAP),
    (dict(cu_new=at(5) + 16), EOVERLAP), (dict(reset=at(12)), EOVERLAP),
])
def test_plan_argument_errors(lib, kw, status):
    assert lib.hlwq_kv_page_plan(ctypes.byref(plan_args(**kw)), None) == status


def test_plan_needs_arguments(lib):
    assert lib.hlwq_kv_page_plan(None, None) == ENULL


def test_packed_arguments_are_the_c_structures():
    assert paged._CACHE.size == ctypes.sizeof(KvCache) and paged._PLAN.size == ctypes.sizeof(KvPlan)
    c = KvCache.from_buffer_copy(paged._CACHE.pack(*range(1, 15)))
    assert [c.k.packed, c.k.norms, c.k.window, c.v.packed, c.v.norms, c.v.window] == [1, 2, 3, 4, 5, 6]
    assert [getattr(c, n) for n, _ in KvCache._fields_[2:]] == list(range(7, 15))
    p = KvPlan.from_buffer_copy(paged._PLAN.pack(*range(1, 20)))
    assert [getattr(p, n) for n, _ in KvPlan._fields_] == list(range(1, 20))


def test_python_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device memory"):
        wq.hlwq_kv_page_plan(i32, i32, i32, i32[:1], i32[:, None], 3)
    with pytest.raises(TypeError, match="tokens"):
        wq.hlwq_kv_page_plan(i32.long(), i32, i32, i32[:1], i32[:, None], 3)
    x = torch.zeros(4, 2, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device memory"):
        wq.hlwq_prompt_attention(x, x, x, i32)
    with pytest.raises(TypeError, match="q must be"):
        wq.hlwq_prompt_attention(x.float(), x, x, i32)
    with pytest.raises(TypeError, match="torch.Tensor"):
        wq.hlwq_prompt_attention(None, x, x, i32)
