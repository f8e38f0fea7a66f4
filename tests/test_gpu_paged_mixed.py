"""GPU tests of paged attention where a step's requests differ: those of few rows and long chunks in one call, so that
both kernels work on it, over more requests than one look of a wave takes in, in exactly the workspace asked for."""
import numpy as np
import pytest

import paged_ref as pr
from test_gpu_paged import Cache, D, bf16_bits, dev16, f64, i32, wq  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FEW = 64  # rows (tokens times query heads of a KV head) up to which a request among others counts as of few rows


def mixed(requests, group, chunks, rng):
    """New tokens of each request: most as many as count as few, some fewer or none, and `chunks` at random places."""
    most = max(FEW // group, 1)
    new = [most if b % 8 else int(rng.integers(0, most + 1)) for b in range(requests)]
    for b, n in zip(rng.permutation(requests), chunks):
        new[b] = n
    return new


@pytest.mark.parametrize("requests,q_heads,kv_heads,bits,page,chunks", [
    (70, 4, 2, 3, 32, [33, 300, 257, 90]),
    (130, 6, 1, 2, 64, [11, 12, 500, 700, 129]),
    (66, 16, 2, 3, 16, [400, 9]),
    (2, 8, 8, 2, 128, [300]),
    (5, 65, 1, 3, 64, [1, 9]),          # a token alone is more than few rows
])
def test_few_rows_and_chunks_in_one_call(wq, requests, q_heads, kv_heads, bits, page, chunks):
    rng = np.random.default_rng(requests)
    group = q_heads // kv_heads
    new = mixed(requests, group, chunks, rng)
    ctx = [int(t) for t in rng.integers(0, 700, requests)]
    n = sum(new)
    assert n * group > FEW * requests  # the call is one of both kernels
    c = Cache(rng, ctx, kv_heads, bits, page, 128, 128)
    q, kv = bf16_bits(rng, n + 3, q_heads, D), [bf16_bits(rng, n + 3, kv_heads, D) for _ in range(2)]
    cu = np.concatenate([[0], np.cumsum(new)])
    need = wq.hlwq_kv_paged_attention_workspace(requests, n + 3, q_heads, kv_heads)
    guard = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((n + 3, q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    wq.hlwq_kv_paged_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), i32(cu), i32([t + m for t, m in zip(ctx, new)]),
                               i32(c.table), *c.tensors(), bits=bits, out=out, workspace=guard[:need])
    torch.cuda.synchronize()
    assert bool((guard[need:] == 0xA5).all())
    got = out.cpu().double().numpy()
    assert np.all(got[n:] == 7.0)
    for b, (t, m) in enumerate(zip(ctx, new)):
        r = slice(cu[b], cu[b + 1])
        k, v = c.tokens_of(b, t, [x[r] for x in kv])
        pr.check_attention(got[r], f64(q[r]), k, v, pr.encoded(t, 128), t, kv_heads)


def test_more_tiles_than_one_dimension_of_a_grid(wq):
    """70,400 tiles of 256 rows, joined by 16 workgroups each: more than 2^20."""
    requests, each, q_heads = 640, 110, 256
    n = requests * each
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(n, h, D, device="cuda", generator=g, dtype=torch.bfloat16) for h in (q_heads, 1, 1))
    cache = Cache(np.random.default_rng(1), [0], 1, 3, 64, 128, 128)
    window = [torch.zeros(requests, 1, 128, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cu = i32(np.arange(requests + 1) * each)
    table = torch.full((requests, 1), -1, dtype=torch.int32, device="cuda")
    out = wq.hlwq_kv_paged_attention(q, k, v, cu, i32([each] * requests), table, *cache.d[:4], *window)
    for b in (0, 300, *range(596, 640)):  # tiles from 65,536 on are those of requests 595 and later
        r = slice(b * each, (b + 1) * each)
        score = (q[r].float().flatten(0, 1) @ k[r, 0].float().T).view(each, q_heads, each) / 16
        score.masked_fill_(torch.ones(each, each, dtype=torch.bool, device="cuda").triu(1)[:, None], -float("inf"))
        p = score.double().softmax(-1)
        o = (p.flatten(0, 1) @ v[r, 0].double()).view(each, q_heads, D)
        # p to bf16 and the output to bf16, 2^-8 each, and the sums in 32 bits (2^-14, as in paged_ref)
        size = (p.flatten(0, 1) @ v[r, 0].double().abs()).view(each, q_heads, D)
        assert bool(((out[r].double() - o).abs() <= (2.0 ** -8 + 2.0 ** -14) * size + 2.0 ** -8 * o.abs()).all()), b
