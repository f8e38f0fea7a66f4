"""Sizes at the limits of the serving operators: what the calls refuse, and what they ask for (CPU only)."""
import weight_quantization_amd as wq

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
