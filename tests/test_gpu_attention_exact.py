"""GPU tests of paged and prompt attention against the definition over the operands that the kernels document, under a bound
that no page, window or partial sum fits into (tests/attention_bound.py): long caches, every window and page size, every
kernel and the joins between them."""
import numpy as np
import pytest

import attention_bound as ab
import paged_ref as pr
from test_gpu_paged import Cache, D, bf16_bits, dev16, f64, i32, strided, wq  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def sides(c, b, held, new):
    """Keys and values of request b, a Side a KV head each; new: the step's bf16 bits, K and V."""
    out = []
    enc = pr.encoded(held, c.residual)
    t, near = np.arange(enc), np.arange(enc, held)
    for i in range(2):
        ids = c.table[b, t // c.page]
        codes = pr.codes_of(c.packed[i][ids, :, t % c.page], c.bits) if enc else np.zeros((0, c.heads, D), int)
        norms = (c.norms[i].view(np.float16)[ids, :, t % c.page].astype(np.float64) if enc else np.zeros((0, c.heads)))
        window = f64(c.window[i][b][:, near % max(c.ring, 1)]) if held > enc else np.zeros((c.heads, 0, D))
        out.append([ab.Side(ab.centroids(codes[:, h], c.bits), norms[:, h], np.concatenate([window[h], f64(new[i][:, h])]))
                    for h in range(c.heads)])
    return out


def some(rng, n, most=24):
    """Rows to look at: the first and last, those beside multiples of 16, and others."""
    if n <= most:
        return None
    near = np.clip(16 * rng.integers(0, n // 16 + 1, 8) + rng.integers(-1, 2, 8), 0, n - 1)
    return np.concatenate([[0, 1, n - 2, n - 1], near, rng.integers(0, n, most - 12)])


def paged(wq, seed, ctx, new, q_heads, kv_heads, bits=3, page=64, residual=128, ring=128, scale=1 / 16, sigma=1.0, extra=0):
    rng = np.random.default_rng(seed)
    c = Cache(rng, ctx, kv_heads, bits, page, residual, ring)
    n = sum(new)
    q, kv = bf16_bits(rng, n, q_heads, D, sigma=sigma), [bf16_bits(rng, n, kv_heads, D) for _ in range(2)]
    cu = np.concatenate([[0], np.cumsum(new)])
    make = (lambda x: strided(x, extra)) if extra else dev16
    out = wq.hlwq_kv_paged_attention(make(q), make(kv[0]), make(kv[1]), i32(cu), i32([t + m for t, m in zip(ctx, new)]),
                                     i32(c.table), *c.tensors(), n_residual=residual, bits=bits, scale=scale)
    got, worst = out.cpu().double().numpy(), 0.0
    for b, (t, m) in enumerate(zip(ctx, new)):
        if m:
            r = slice(cu[b], cu[b + 1])
            worst = max(worst, ab.check(got[r], f64(q[r]), *sides(c, b, t, [x[r] for x in kv]), t, some(rng, m), scale))
    print(f"largest error {worst:.3f} of its bound", flush=True)


@pytest.mark.parametrize("ctx,new", [
    ([0], [1]), ([1], [1]), ([129], [1]), ([500], [1]), ([2049], [1]), ([5000], [1]), ([9000], [1]),
    ([0, 1, 15, 128, 129, 144, 145, 192, 193, 1000, 3000], [1] * 11), ([1000, 30], [5, 6]), ([4000, 0, 999], [3, 1, 0]),
])
@pytest.mark.parametrize("q_heads,kv_heads,bits,page", [(24, 4, 3, 64), (6, 2, 2, 16)])
def test_few_rows(wq, ctx, new, q_heads, kv_heads, bits, page):
    paged(wq, sum(ctx) + len(new), ctx, new, q_heads, kv_heads, bits, page)


@pytest.mark.parametrize("ctx,new,q_heads,kv_heads,bits,page,residual,ring", [
    ([3000], [300], 24, 4, 3, 64, 128, 128), ([4099], [130], 16, 2, 2, 16, 128, 300), ([9000], [200], 2, 1, 3, 64, 128, 128),
    ([2000, 700, 0], [101, 257, 64], 6, 2, 3, 256, 0, 0), ([900], [33], 1, 1, 3, 32, 200, 201),
    ([1000, 1000], [65, 64], 8, 8, 2, 128, 37, 37), ([333], [257], 1, 1, 2, 64, 128, 128), ([0], [300], 6, 1, 3, 64, 128, 128),
])
def test_chunks(wq, ctx, new, q_heads, kv_heads, bits, page, residual, ring):
    paged(wq, sum(new), ctx, new, q_heads, kv_heads, bits, page, residual, ring, extra=8)


@pytest.mark.parametrize("residual,ring", [(0, 0), (1, 1), (37, 37), (64, 100), (128, 1000), (600, 600)])
@pytest.mark.parametrize("bits,page,new", [(3, 16, [1, 1, 1]), (2, 256, [3, 1, 2]), (3, 128, [20, 90, 133])])
def test_windows(wq, residual, ring, bits, page, new):
    paged(wq, residual + ring, [1555, 38, 300], new, 12, 2, bits, page, residual, ring)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (8, 8), (8, 1), (10, 2), (17, 1), (64, 2)])
@pytest.mark.parametrize("new", [[2, 1], [40, 50]])
def test_heads(wq, q_heads, kv_heads, new):
    paged(wq, q_heads, [2500, 133], new, q_heads, kv_heads, 3 if q_heads % 2 else 2)


@pytest.mark.parametrize("scale,sigma", [(1 / 16, 8.0), (1.0, 0.01), (-0.05, 1.0), (0.0, 1.0), (1 / 16, 300.0)])
@pytest.mark.parametrize("new", [[2, 1], [90, 130]])
def test_scales(wq, scale, sigma, new):
    paged(wq, 5, [1900, 270], new, 6, 1, scale=scale, sigma=sigma)


def test_few_rows_and_chunks_over_many_requests(wq):
    rng = np.random.default_rng(70)
    ctx = [int(t) for t in rng.integers(0, 2500, 70)]
    new = [int(rng.integers(0, 33)) for _ in range(70)]
    new[7], new[40], new[69] = 900, 400, 300
    assert 2 * sum(new) > 64 * 70
    paged(wq, 71, ctx, new, 4, 2)


@pytest.mark.parametrize("lens,q_heads,kv_heads", [
    # tiles of 128 rows
    ([70], 6, 1), ([383], 24, 4), ([300] * 8, 6, 1), ([2800], 24, 4), ([1, 2, 33, 64, 0, 65, 250], 4, 2), ([1500] * 4, 24, 4),
    ([2500, 3, 1200, 800, 1, 2000], 16, 2),
    # their keys halved
    ([384], 24, 4), ([700], 6, 1), ([1500], 24, 4), ([513, 300, 400], 5, 1),
    # tiles of 256 rows
    ([150] * 65, 16, 8), ([7000], 24, 4),
])
def test_prompts(wq, lens, q_heads, kv_heads):
    rng = np.random.default_rng(sum(lens))
    n = sum(lens)
    q, kv = bf16_bits(rng, n, q_heads, D), [bf16_bits(rng, n, kv_heads, D) for _ in range(2)]
    cu = np.concatenate([[0], np.cumsum(lens)])
    got = wq.hlwq_prompt_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), i32(cu)).cpu().double().numpy()
    none, worst = np.zeros((0, D)), 0.0
    for b, m in enumerate(lens):
        if m:
            r = slice(cu[b], cu[b + 1])
            k, v = ([ab.Side(none, np.zeros(0), f64(x[r][:, h])) for h in range(kv_heads)] for x in kv)
            worst = max(worst, ab.check(got[r], f64(q[r]), k, v, 0, some(rng, m, 20)))
    print(f"largest error {worst:.3f} of its bound", flush=True)
