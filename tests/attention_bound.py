"""A bound on what attention over codes may be off by that leaves no room for a page, a window or a token left out.

The definition with the operands that the kernels document: centroids rounded to fp16, the rotated query rounded to fp16
over a power of two, everything else exact, in 64 bits.  What a kernel may differ by from that is counted below; it comes
to 0.015 to 0.03 of a row over 500 to 5000 tokens.  (The bound of paged_ref is against the definition itself and takes
those two roundings as errors of any sign in every score: 0.15 to 1.3 rows.)

With scores off by d_j and the weights' products by e_j, a row off by  sum_j p_j (exp(d_j) - 1) (v_j - o) / sum_j p_j
exp(d_j)  +  sum_j p_j e_j v_j :  a score's error moves the row only by how far its value lies from the row.

  d_j   256 products summed in fp32, 2^-23 each whatever the matrix unit's rounding: 2^-15 sum_d |q_d k_jd|;
        where the query's rotation in fp32 (eight levels, 2^-24 each) may fall on the other side of an fp16 rounding, the
        step between the two; norm, factor, argument and exponential: 2^-21 of the scores' size; raises of the running
        maximum and joins of partial sums: 2^-16.
  e_j   the weight's rounding: fp16 2^-11 where encoded (with an absolute 2^-31 of the largest norm's, for weights that
        are subnormal beside it), bf16 2^-8 elsewhere; fp32 sums over tokens, (T / 32 + 64) 2^-23, weights' sum T 2^-24.
  row   2^-8, rounded to bf16.
"""
import numpy as np

import paged_ref as pr

D = 256
H = pr.hadamard()


def rotated(q):
    """H q of bf16 rows [.., 256] as the kernels carry it, rounded to fp16 over a power of two; and by how much each of
    its values may differ from that."""
    x = q @ H
    e = np.frexp(np.abs(x).max(-1, keepdims=True))[1] - 1
    y = np.ldexp(x, -e)
    err = np.ldexp(9 * 2.0 ** -24 * np.abs(q).sum(-1, keepdims=True), -e)

    def half(a):
        return a.astype(np.float16).astype(np.float64)

    r = half(y)
    step = np.maximum(np.abs(half(y + err) - r), np.abs(half(y - err) - r))
    return np.ldexp(r, e), np.ldexp(step, e)


def centroids(codes, bits):
    """The fp16 centroids of codes, in 64 bits."""
    return pr.lm.table(bits)[0].astype(np.float32).astype(np.float16).astype(np.float64)[codes]


class Side:
    """Keys or values of one request and KV head: centroids [enc, 256] and norms [enc] of the encoded tokens, then the
    vectors [m, 256] of the others."""

    def __init__(self, cent, norms, near):
        self.cent, self.norms, self.near = cent, norms, near
        old = (cent @ H) * (norms / D)[:, None] if len(norms) else np.zeros((0, D))
        self.vectors = np.concatenate([old, near])


def expect(q, k, v, seen, scale=1 / 16):
    """Rows q [rows, 256] of which row i sees the first seen[i] tokens: the outputs, and a bound on the 2-norm of each
    row's error."""
    enc, total = len(k.norms), len(k.vectors)
    s = np.empty((len(q), total))
    d = np.empty_like(s)
    if enc:
        qr, step = rotated(q)
        s[:, :enc] = scale * (qr @ k.cent.T) * (k.norms / D)
        d[:, :enc] = abs(scale) * ((step + 2.0 ** -15 * np.abs(qr)) @ np.abs(k.cent).T) * (k.norms / D)
    s[:, enc:] = scale * (q @ k.near.T)
    d[:, enc:] = abs(scale) * 2.0 ** -15 * (np.abs(q) @ np.abs(k.near).T)
    there = np.arange(total) < np.asarray(seen)[:, None]
    largest = np.where(there, np.abs(s), 0).max(-1, keepdims=True)
    d += 2.0 ** -21 * (np.abs(s) + largest + 1) + 2.0 ** -16
    s = np.where(there, s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    o = p @ v.vectors
    size = np.linalg.norm(v.vectors, axis=-1)
    apart = np.sqrt(np.maximum(size ** 2 - 2 * (o @ v.vectors.T) + (o * o).sum(-1, keepdims=True), 0))
    off = np.where(there, p * np.expm1(d) * apart, 0).sum(-1) / np.where(there, p * np.exp(-d), 0).sum(-1)
    rounding = np.where(np.arange(total) < enc, 2.0 ** -11, 2.0 ** -8) + (total / 32 + 64) * 2.0 ** -23
    off += (p * rounding * size).sum(-1)
    if enc:
        off += enc * 2.0 ** -31 * size[:enc].max()
    return o, off + (2.0 ** -8 + total * 2.0 ** -24) * np.linalg.norm(o, axis=-1)


def check(out, q, keys, values, base, rows=None, scale=1 / 16):
    """out, q [rows, q_heads, 256] of one request in 64 bits; keys, values: a Side a KV head; row i sees base + i + 1 tokens.
    rows: those to look at (all by default).  Returns the largest error over its bound."""
    g = q.shape[1] // len(keys)
    rows = np.arange(len(q)) if rows is None else np.unique(np.asarray(rows))
    worst = 0.0
    for h, (k, v) in enumerate(zip(keys, values)):
        heads = slice(h * g, (h + 1) * g)
        o, bound = expect(q[rows, heads].reshape(-1, D), k, v, np.repeat(base + rows + 1, g), scale)
        err = np.linalg.norm(out[rows, heads].reshape(-1, D) - o, axis=-1)
        ok = err <= bound
        assert np.all(ok), f"KV head {h}: rows {rows[np.where(~ok)[0][:4] // g]}, error {err[~ok][:4]}, bound {bound[~ok][:4]}"
        worst = max(worst, float((err / np.maximum(bound, 1e-300)).max()))
    return worst
