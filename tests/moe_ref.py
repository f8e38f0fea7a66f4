"""The mixture-of-experts layer from its definition in 64 bits, with a bound on what the kernels may differ by.

The definition takes the operands that the kernels document (centroids rounded to fp16; a token's activations rotated in
fp32 and rounded to fp16 over a power of two), everything else exact.  What is left is counted per output:

  preactivations  fp32 sums of `hidden` products, 2^-23 each whatever the matrix unit's rounding, of the sum of sizes;
  inner values    the activation's slope, at most 1.2, times that; its exponential's argument, division and products:
                  2^-20 (1 + |z|) of the value for an argument z;
  rotated again   a block's errors add up; eight fp32 roundings of 2^-24; fp16 2^-11 of the value, or half a step of the
                  smallest fp16 over the row's power of two;
  output          fp32 sums as above, and 2^-8, rounded to bf16.
"""
import numpy as np

import paged_ref as pr
from oracle import lloyd_max as lm

B = 128
H = pr.hadamard(B)


def f32_of(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def codes_of(packed, bits):
    bit = np.unpackbits(packed, axis=-1, bitorder="little").reshape(*packed.shape[:-1], B, bits)
    return (bit * (1 << np.arange(bits))).sum(-1)


def centroids(packed, bits):
    """fp16 centroids [.., out, nb, 128] of packed codes, in 64 bits."""
    return lm.table(bits)[0].astype(np.float32).astype(np.float16).astype(np.float64)[codes_of(packed, bits)]


def blocks(x):
    """Rows [.., n] as zero-padded blocks [.., nb, 128]."""
    nb = -(-x.shape[-1] // B)
    y = np.zeros((*x.shape[:-1], nb * B), x.dtype)
    y[..., :x.shape[-1]] = x
    return y.reshape(*x.shape[:-1], nb, B)


def exponent(top):
    """The power of two that a row is taken over."""
    return np.where(top > 0, np.maximum(np.frexp(top)[1] - 1, -110), 0)


def rotated(x):
    """Rotated rows of fp32 [.., n] as the kernels carry them, [.., nb, 128] in 64 bits: butterflies in fp32, fp16."""
    e = exponent(np.abs(x).max(-1, initial=0))[..., None, None]
    y = np.ldexp(blocks(x.astype(np.float32)), 7 - e).astype(np.float32)
    h = 1
    while h < B:
        y = y.reshape(*y.shape[:-1], B // (2 * h), 2, h) if y.shape[-1] == B else y
        a, b = y[..., 0, :], y[..., 1, :]
        y = np.stack([a + b, a - b], -2).reshape(*x.shape[:-1], -1, B)
        h *= 2
    return np.ldexp(y.astype(np.float16).astype(np.float64), e - 7)


def product(cent, norms, x, dx):
    """Rows [out, nb, 128] of centroids times norms / 128 over blocks x [t, nb, 128] with errors dx: [t, out] and its
    error's bound."""
    s = norms.astype(np.float64) / B
    out, nb, _ = cent.shape
    w = (cent * s[..., None]).reshape(out, nb * B)
    x, dx = x.reshape(len(x), -1), dx.reshape(len(x), -1)
    return x @ w.T, dx @ np.abs(w).T + (nb * B + 8) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)


def act(g, kind):
    z = g if kind == "silu" else np.sqrt(2 / np.pi) * 2 * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-z)), 2.0 ** -20 * (1 + np.abs(z))


def experts(x, ids, weights, up, down, bits, kind):
    """x fp32 values of bf16 [tokens, hidden], ids and weights [tokens, k], up and down (packed, norms): outputs
    [tokens, hidden] in 64 bits and a bound on each one's error before its rounding to bf16."""
    tokens, hidden = x.shape
    inner = up[0].shape[1] // 2
    xr = rotated(x)
    y, dy = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    for e in np.unique(ids):
        if not 0 <= e < up[0].shape[0]:
            continue
        t, j = np.nonzero(ids == e)
        a, da = product(centroids(up[0][e], bits), up[1][e], xr[t], np.zeros_like(xr[t]))
        g, rel = act(a[:, :inner], kind)
        u, w = a[:, inner:], weights[t, j].astype(np.float64)[:, None]
        h = g * u * w
        dh = np.abs(w) * (1.2 * da[:, :inner] * (np.abs(u) + da[:, inner:]) + np.abs(g) * da[:, inner:]) + rel * np.abs(h)
        hb, db = blocks(h), blocks(dh)
        hr = hb @ H
        scale = np.ldexp(1.0, exponent(np.abs(h).max(-1, initial=0)) - 7)[:, None, None]
        dr = (db.sum(-1) + 8 * 2.0 ** -24 * np.abs(hb).sum(-1))[..., None] * (1 + 2.0 ** -10)
        dr = dr + 2.0 ** -11 * np.abs(hr) + 2.0 ** -25 * 2 * scale
        o, do = product(centroids(down[0][e], bits), down[1][e], hr, dr)
        np.add.at(y, t, o)
        np.add.at(dy, t, do + ids.shape[1] * 2.0 ** -23 * np.abs(o))
    return y, dy


def check(out, y, dy):
    bound = dy + 2.0 ** -8 * (np.abs(y) + dy)
    err = np.abs(out - y)
    ok = err <= bound
    assert np.all(ok), f"{np.argwhere(~ok)[:4].tolist()}: error {err[~ok][:4]}, bound {bound[~ok][:4]}"
    return float((err / np.maximum(bound, 1e-300)).max(initial=0))


def route(x, router, k, renormalize):
    """The k best experts of each token and their weights, in 64 bits; ties to the lower index."""
    logits = x.astype(np.float64) @ router.astype(np.float64).T
    ids = np.argsort(-logits, -1, kind="stable")[:, :k]
    top = np.take_along_axis(logits, ids, -1)
    high = logits.max(-1, keepdims=True)
    w = np.exp(top - high)
    return ids, w / (w if renormalize else np.exp(logits - high)).sum(-1, keepdims=True)
