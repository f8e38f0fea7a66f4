"""Sizes at the limits of the serving operators: what the calls refuse, and what they ask for (CPU only).

A call that must not be refused for its sizes is made with a workspace of no bytes, so that it ends there and launches
nothing.
"""
import pytest

import weight_quantization_amd as wq
from test_paged_host import EALIGN, ELIMIT, ESHAPE, append, at, attention, cache, lib, prompt  # noqa: F401

SPLIT_TILE = 2 * 16 * (256 + 2) * 4   # bytes of workspace of a tile of 16 rows
SPLIT = 512 * SPLIT_TILE
CHUNK = 512 * 256 * (256 + 2) * 4


def test_workspace_of_a_few_long_requests_does_not_grow_with_their_rows():
    w = wq.hlwq_kv_paged_attention_workspace
    # two requests: at most four tiles of 16 rows each and KV head belong to requests of up to 64 rows
    assert w(2, 8192, 24, 4) == w(2, 16384, 24, 4) == w(2, 10 ** 6, 24, 4) <= SPLIT + 2 * 4 * 4 * SPLIT_TILE + CHUNK
    assert w(2, 16384, 32, 8) <= SPLIT + 2 * 4 * 8 * SPLIT_TILE + CHUNK
    # one request, or heads of which one token has more than 64 rows: the chunk kernel's alone
    assert w(1, 16384, 24, 4) == w(2, 16384, 65, 1) == CHUNK
    # requests of few rows: as many tiles as whole ones fill, and one more a request and KV head
    assert w(64, 64, 24, 4) == SPLIT + (64 * 6 // 16 + 64) * 4 * SPLIT_TILE


def sized(lib, requests, rows, q_heads, kv_heads, width=0, page=64):
    """The status of a paged attention call of these sizes with no workspace: ESHAPE unless the sizes are refused."""
    c = cache(requests=requests, kv_heads=kv_heads, page_size=page, n_residual=0, ring=0)
    return attention(lib, c, qs=256 * q_heads, hq=q_heads, ks=256 * kv_heads, vs=256 * kv_heads, width=width, rows=rows,
                     bytes_=0)


@pytest.mark.parametrize("requests,rows,q_heads,kv_heads,refused", [
    (1, 1, 24, 4, False), (64, 64, 24, 4, False), (2, 10 ** 6, 24, 4, False), (1, 10 ** 7, 24, 4, False),
    (2, 720_000, 24, 4, False),                       # over a million tiles of 16 rows, all the chunk kernel's
    (1, 2 ** 31 // 24 - 1, 24, 24, False),            # the most rows there are, in one request
    (2 ** 20, 2 ** 31 // 4096 - 1, 4096, 1, False),
    (2 ** 20, 2 ** 20 - 1, 1, 1, False),              # 2^20 - 1 tiles: one a token
    (2 ** 20, 2 ** 20, 1, 1, True),
    (2 ** 18, 2 ** 18, 32, 8, True),
    (2 ** 17 + 1, 2 ** 25, 8, 4, True),               # chunks, but 4 tiles of each request may be the split kernel's
    (2 ** 16 - 1, 2 ** 25, 8, 4, False),
])
def test_the_workspace_is_none_for_sizes_that_are_refused_and_only_for_those(lib, requests, rows, q_heads, kv_heads, refused):
    assert sized(lib, requests, rows, q_heads, kv_heads) == (ELIMIT if refused else ESHAPE)
    need = wq.hlwq_kv_paged_attention_workspace(requests, rows, q_heads, kv_heads)
    assert need == 0 if refused else need >= min(SPLIT, CHUNK)


def test_tables_too_wide_for_the_tiles_are_refused(lib):
    # T tiles, of page_size * width / 128 blocks each
    assert sized(lib, 1, 1, 4, 4, width=2 ** 20, page=256) == ESHAPE        # 4 * 2^21
    assert sized(lib, 256, 256, 4, 4, width=2 ** 20, page=256) == ELIMIT    # 1024 * 2^21
    assert sized(lib, 256, 255, 4, 4, width=2 ** 20, page=256) == ESHAPE
    assert sized(lib, 1, 10 ** 6, 4, 4, width=2 ** 20, page=256) == ESHAPE  # none of the split kernel's
    assert sized(lib, 63, 10 ** 6, 4, 4, width=2 ** 20, page=256) == ESHAPE   # 63 * 4 * 4 = 1008 tiles
    assert sized(lib, 64, 10 ** 6, 4, 4, width=2 ** 20, page=256) == ELIMIT   # 1024


@pytest.mark.parametrize("kv_heads,rows,status", [(1, 2 ** 29 - 32, EALIGN), (1, 2 ** 29 - 31, ELIMIT), (8, 2 ** 26 - 4, EALIGN),
                                                  (8, 2 ** 26 - 3, ELIMIT), (4096, 2 ** 31 - 1, ELIMIT)])
def test_an_append_past_one_launch_is_refused(lib, kv_heads, rows, status):
    # (keys 8 bytes off their place end the calls whose sizes are taken)
    stride = 256 * kv_heads
    assert append(lib, cache(kv_heads=kv_heads), k=at(6) + 8, ks=stride, vs=stride, rows=rows) == status


@pytest.mark.parametrize("rows,n,kv_heads,status", [(2 ** 20, 2 ** 20, 8, ELIMIT), (2 ** 20, 2 ** 20, 7, EALIGN),
                                                    (2 ** 22, 2, 24, EALIGN), (2 ** 18, 2 ** 18, 33, ELIMIT)])
def test_a_prompt_call_past_one_launch_is_refused(lib, rows, n, kv_heads, status):
    w = 256 * kv_heads
    assert prompt(lib, qs=w, ks=w, vs=w, n=n, rows=rows, hq=kv_heads, hk=kv_heads, q=at(0) + 8 * (status == EALIGN)) == status
