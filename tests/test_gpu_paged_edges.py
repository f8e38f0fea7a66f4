"""GPU tests of the serving operators at values that lengths and queries may take but hardly ever do."""
import numpy as np
import pytest

from test_gpu_paged import Cache, D, bf16_bits, dev16, i32, wq  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# few rows of one request, many of one, and both at once
STEPS = [[5], [300], [2, 200]]


@pytest.mark.parametrize("new", STEPS)
def test_lengths_far_below_the_new_tokens(wq, new):
    """Any length below a request's new tokens counts as equal to them, those whose difference passes 32 bits too."""
    rng = np.random.default_rng(len(new))
    n = len(new)
    c = Cache(rng, [700] * n, 2, 3, 64, 128, 128)  # pages and a window that the step must not see
    q, k, v = (dev16(bf16_bits(rng, sum(new), h, D)) for h in (4, 2, 2))
    cu = i32(np.concatenate([[0], np.cumsum(new)]))
    want = wq.hlwq_kv_paged_attention(q, k, v, cu, i32(new), i32(c.table), *c.tensors())
    assert bool(torch.isfinite(want).all())
    for low in (0, -1, -2 ** 30, 1 - 2 ** 31, -2 ** 31):
        got = wq.hlwq_kv_paged_attention(q, k, v, cu, i32([low] * n), i32(c.table), *c.tensors())
        assert torch.equal(got, want), low


@pytest.mark.parametrize("new", STEPS)
def test_queries_near_the_smallest(wq, new):
    """Queries below 2^-118, subnormal ones among them: no score of theirs differs from 0 by what a weight could hold, so
    that the rows are those of queries of zero."""
    rng = np.random.default_rng(10 + len(new))
    n, rows = len(new), sum(new)
    c = Cache(rng, [700] * n, 2, 3, 64, 128, 128)
    k, v = (dev16(bf16_bits(rng, rows, 2, D)) for _ in range(2))
    cu, lens = i32(np.concatenate([[0], np.cumsum(new)])), i32([700 + m for m in new])
    zero = torch.zeros(rows, 4, D, dtype=torch.bfloat16, device="cuda")
    want = wq.hlwq_kv_paged_attention(zero, k, v, cu, lens, i32(c.table), *c.tensors())
    for top in (0x0001, 0x0002, 0x0010, 0x007F, 0x0080, 0x0400):
        bits = rng.integers(0, top + 1, (rows, 4, D)) | (rng.integers(0, 2, (rows, 4, D)) << 15)
        bits[0] = 0
        bits[0, 1, 7] = top  # one value alone
        got = wq.hlwq_kv_paged_attention(dev16(bits.astype(np.uint16)), k, v, cu, lens, i32(c.table), *c.tensors())
        assert torch.equal(got, want), hex(top)


@pytest.mark.parametrize("new", STEPS)
def test_queries_of_any_size(wq, new):
    """q times 2^s under a scale over 2^s: powers of two pass through every product, sum and rounding, so the outputs are
    the same bits, also where a sum of 256 of the queries' values passes fp32 (s = 118: 256 times 4 times 2^118)."""
    rng = np.random.default_rng(20 + len(new))
    n, rows = len(new), sum(new)
    c = Cache(rng, [700] * n, 2, 3, 64, 128, 128)
    k, v = (dev16(bf16_bits(rng, rows, 2, D)) for _ in range(2))
    cu, lens = i32(np.concatenate([[0], np.cumsum(new)])), i32([700 + m for m in new])
    q = rng.integers(-16, 17, (rows, 4, D)) / 4.0
    q[0], q[-1, 2] = 4.0, -4.0
    q = torch.from_numpy(q).cuda()
    want = wq.hlwq_kv_paged_attention(q.to(torch.bfloat16), k, v, cu, lens, i32(c.table), *c.tensors())
    assert bool(torch.isfinite(want).all())
    for s in (-90, -20, 60, 118):
        got = wq.hlwq_kv_paged_attention((q * 2.0 ** s).to(torch.bfloat16), k, v, cu, lens, i32(c.table), *c.tensors(),
                                         scale=2.0 ** (-4 - s))
        assert torch.equal(got, want), s
