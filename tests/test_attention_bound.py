"""What tests/attention_bound.py lets pass and what it does not (CPU only): the arithmetic of the kernels, carried out in
32 and 16 bits here, passes; a row without its window, without a page or without the token it attends to most does not."""
import numpy as np
import pytest

import attention_bound as ab
import paged_ref as pr

D = 256
LENGTHS = [500, 900, 2049, 3000, 5000]


def bf16(x):
    u = np.asarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).view(np.float32)


def make(rng, held, new, bits=3, residual=128, sigma=1.0, group=6):
    """q [new * group, 256], keys and values of a request of random codes and unit normal vectors, seen of each row."""
    enc = max(held - residual, 0)
    sides = [ab.Side(ab.centroids(rng.integers(0, 1 << bits, (enc, D)), bits),
                     rng.uniform(8, 24, enc).astype(np.float16).astype(np.float64),
                     bf16(rng.standard_normal((held - enc + new, D))).astype(np.float64)) for _ in range(2)]
    q = bf16(rng.standard_normal((new * group, D)) * sigma).astype(np.float64)
    return q, *sides, np.repeat(held + 1 + np.arange(new), group)


def kernel(q, k, v, seen, scale=1 / 16, block=128):
    """The kernels' arithmetic: fp32 sums, an online softmax over blocks of tokens, weights rounded to 16 bits."""
    f32, enc = np.float32, len(k.norms)
    r, _ = ab.rotated(q)
    top = np.ldexp(1.0, np.frexp(v.norms.max())[1] - 7) if enc else 1.0
    m, l = np.full((len(q), 1), -np.inf, f32), np.zeros((len(q), 1), f32)
    o = [np.zeros((len(q), D), f32) for _ in range(2)]  # over centroids, over vectors
    cuts = sorted({*range(0, enc, block), enc, *range(enc, len(k.vectors), block), len(k.vectors)})
    for a, b in zip(cuts, cuts[1:]):
        old = b <= enc
        if old:
            s = (r.astype(f32) @ k.cent[a:b].T.astype(f32)) * k.norms[a:b].astype(f32) * f32(scale / D)
        else:
            s = (q.astype(f32) @ k.near[a - enc:b - enc].T.astype(f32)) * f32(scale)
        s = np.where(np.arange(a, b) < seen[:, None], s, f32(-np.inf))
        mn = np.maximum(m, s.max(-1, keepdims=True))
        f = np.exp(m - mn)
        p = np.exp(s - mn)
        m, l, o = mn, l * f + p.sum(-1, keepdims=True), [x * f for x in o]
        if old:
            w = (p * (v.norms[a:b] / top).astype(f32)).astype(np.float16).astype(f32)
            o[0] += w @ v.cent[a:b].astype(f32)
        else:
            o[1] += bf16(p) @ v.near[a - enc:b - enc].astype(f32)
    return bf16((o[0] @ ab.H.astype(f32) * f32(top / D) + o[1]) / l).astype(np.float64)


def without(q, k, v, seen, keep, scale=1 / 16):
    """The rows of the tokens `keep` alone, rounded to bf16."""
    s = np.where((np.arange(len(keep)) < seen[:, None]) & keep, scale * (q @ k.vectors.T), -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    return bf16(p / p.sum(-1, keepdims=True) @ v.vectors).astype(np.float64)


def ratio(out, o, bound):
    return np.linalg.norm(out - o, axis=-1) / bound


@pytest.mark.parametrize("held", [0, 1, 100, 129, *LENGTHS])
@pytest.mark.parametrize("bits", [3, 2])
@pytest.mark.parametrize("sigma", [1.0, 0.05, 8.0, 300.0])
def test_the_kernels_arithmetic_passes(held, bits, sigma):
    rng = np.random.default_rng(held + bits)
    q, k, v, seen = make(rng, held, 3, bits, sigma=sigma)
    o, bound = ab.expect(q, k, v, seen)
    assert ratio(kernel(q, k, v, seen), o, bound).max() <= 1


@pytest.mark.parametrize("held", LENGTHS)
@pytest.mark.parametrize("bits", [3, 2])
def test_what_is_left_out_does_not_pass(held, bits):
    rng = np.random.default_rng(held + bits)
    q, k, v, seen = make(rng, held, 2, bits)
    enc, total = len(k.norms), len(k.vectors)
    o, bound = ab.expect(q, k, v, seen)
    assert (ratio(0 * o, o, bound) > 8).all()
    at = np.arange(total)
    # the window, a page of 64 tokens (the first, one in the middle, the last whole one), half a page: most rows show it
    for gone in ((at >= enc) & (at < held), at < 64, (at >= 192) & (at < 256),
                 (at >= enc // 64 * 64 - 64) & (at < enc // 64 * 64), (at >= 128) & (at < 160)):
        assert (ratio(without(q, k, v, seen, ~gone), o, bound) > 1).mean() > 0.5, (held, gone.sum())
    # another page's keys in a page's place
    other = ab.Side(k.cent.copy(), k.norms, k.near)
    other.vectors[64:128] = k.vectors[128:192]
    assert (ratio(without(q, other, v, seen, at >= 0), o, bound) > 1).mean() > 0.5


@pytest.mark.parametrize("held", [0, 500, 5000])
def test_the_token_attended_to_most_must_be_there(held):
    rng = np.random.default_rng(held)
    q, k, v, seen = make(rng, held, 5, sigma=3.0, group=1)
    o, bound = ab.expect(q, k, v, seen)
    s = np.where(np.arange(len(k.vectors)) < seen[:, None], q @ k.vectors.T, -np.inf)
    for i in range(1 if held == 0 else 0, len(q)):  # (the only token of a row cannot be left out)
        keep = np.arange(len(k.vectors)) != s[i].argmax()
        assert ratio(without(q[i:i + 1], k, v, seen[i:i + 1], keep), o[i:i + 1], bound[i:i + 1])[0] > 1


def test_large_queries_see_the_right_token():
    rng = np.random.default_rng(3)
    q, k, v, seen = make(rng, 900, 3, sigma=300.0)
    o, bound = ab.expect(q, k, v, seen)
    assert (ratio(0 * o, o, bound) > 1).mean() > 0.9
    assert (ratio(v.vectors[rng.integers(0, 900, len(q))], o, bound) > 1).mean() > 0.9


@pytest.mark.parametrize("n", [70, 517, 1500])
def test_prompts(n):
    rng = np.random.default_rng(n)
    q, k, v, seen = make(rng, 0, n, group=1)
    o, bound = ab.expect(q, k, v, seen)
    assert ratio(kernel(q, k, v, seen, block=64), o, bound).max() <= 1
    at = np.arange(n)
    keep = ~((at >= 32) & (at < 64))
    late = at >= 64
    assert (ratio(without(q, k, v, seen, keep), o, bound)[late] > 1).mean() > 0.5
    # a row that sees one token too few or too many
    assert (ratio(without(q, k, v, np.maximum(seen - 1, 1), at >= 0), o, bound)[1:64] > 1).mean() > 0.5
    assert (ratio(without(q, k, v, np.minimum(seen + 1, n), at >= 0), o, bound)[:64] > 1).mean() > 0.5


def test_rotation_in_32_bits_stays_within_its_slack():
    rng = np.random.default_rng(0)
    q = bf16(rng.standard_normal((64, D)) * np.exp(rng.uniform(-20, 20, (64, 1)))).astype(np.float64)
    r, step = ab.rotated(q)
    for order in ((1, 2, 4, 8, 16, 32, 64, 128), (1, 2, 4, 16, 32, 64, 128, 8)):  # the two kernels'
        x = q.astype(np.float32)
        for h in order:
            y = x.reshape(64, D // (2 * h), 2, h)
            x = np.stack((y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]), 2).reshape(64, D)
        e = np.frexp(np.abs(x).max(-1, keepdims=True))[1] - 1
        got = np.ldexp(np.ldexp(x, -e).astype(np.float16).astype(np.float64), e)
        assert (np.abs(got - r) <= step).all()
    assert (step == 0).mean() > 0.9
    assert np.abs(r - q @ pr.hadamard()).max() <= (2.0 ** -11 * np.abs(q @ pr.hadamard()).max(-1)).max()
