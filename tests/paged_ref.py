"""Plain CPU forms of the paged-cache operators, for the tests: the page plan and
the append step by step in Python (codes from the oracle), attention in 64 bits
straight from its definition.  Shares no code with the package.
"""
import math

import numpy as np

from oracle import hlwq_ref as ref
from oracle import lloyd_max as lm

D = 256


def encoded(tokens, residual):
    return max(tokens - residual, 0)


def plan(tokens, n_new, reset, stack, n_free, table, rows, page, residual):
    """One step's plan; stack and table are changed in place.  Returns (cu, lens,
    row_request, positions, slots, n_free, status)."""
    B, width, pool = len(tokens), table.shape[1], len(stack)
    row_request, positions, slots = (np.full(rows, -1, np.int32) for _ in range(3))

    def pages(t):
        return -(-encoded(t, residual) // page)

    held = [0 if r else t for t, r in zip(tokens, reset)]
    want = [pages(h + n) if n >= 0 and h >= 0 else 0 for h, n in zip(held, n_new)]
    had = [pages(h) for h in held]
    back = [int(p) for b in range(B) if reset[b] for p in table[b, :pages(tokens[b])]]
    bad = (min([0, *tokens, *n_new]) < 0 or sum(n_new) > rows or not 0 <= n_free <= pool or n_free + len(back) > pool
           or max([0, *want, *(pages(t) for t in tokens)]) > width or any(not 0 <= p < pool for p in back)
           or any(h + n > 2 ** 31 - 1 for h, n in zip(held, n_new)))
    need = sum(w - h for w, h in zip(want, had))
    top = n_free + len(back)
    if bad or need > top:
        return (np.zeros(B + 1, np.int32), np.array(tokens, np.int32), row_request, positions, slots, n_free,
                -1 if bad else need - top)
    stack[n_free:top] = back
    cu = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
    for b in range(B):
        for p in range(had[b], want[b]):
            top -= 1
            table[b, p] = stack[top]
        for i in range(n_new[b]):
            row, t = cu[b] + i, held[b] + i
            row_request[row], positions[row] = b, t
            if t >= residual:
                old = t - residual
                slots[row] = table[b, old // page] * page + old % page
    lens = np.array([h + n for h, n in zip(held, n_new)], np.int32)
    return cu, lens, row_request, positions, slots, top, 0


def append(new, cu, lens, row_request, slots, packed, norms, window, residual, bits):
    """A step's rows of keys or values (bf16 bits [rows, heads, 256]) into packed u8 [pages, heads, page, 32 bits],
    norms u16 and window u16 [requests, heads, ring, 256], in place."""
    page, ring, heads = packed.shape[2], window.shape[2], packed.shape[1]
    before = window.copy()
    leaving = []
    for row, b in enumerate(row_request):
        if b < 0:
            continue
        n = int(cu[b + 1] - cu[b])
        held = int(lens[b]) - n
        t = held + row - int(cu[b])
        if slots[row] >= 0:
            old = t - residual
            leaving.append((slots[row], before[b, :, old % ring] if old < held else new[row - residual]))
        if t >= lens[b] - residual:
            window[b, :, t % ring] = new[row]
    if leaving:
        src = np.stack([v for _, v in leaving])  # [m, heads, 256]
        p, n16 = ref.kv_quantize_c(np.ascontiguousarray(src[None]), n_residual=0, bits=bits)
        for (slot, _), c, n in zip(leaving, p[0], n16[0]):
            packed[slot // page, :, slot % page] = c
            norms[slot // page, :, slot % page] = n.view(np.uint16)


def hadamard(n=D):
    h = np.ones((1, 1))
    while h.shape[0] < n:
        h = np.block([[h, h], [h, -h]])
    return h


def codes_of(packed, bits):
    """Codes [.., 256] of packed bytes [.., 32 bits], bit by bit."""
    bit = np.unpackbits(packed, axis=-1, bitorder="little").reshape(*packed.shape[:-1], D, bits)
    return (bit * (1 << np.arange(bits))).sum(-1)


def decoded(packed, norms, bits):
    """The vectors that codes and norms stand for, in 64 bits."""
    cent, _ = lm.table(bits)
    return cent.astype(np.float64)[codes_of(packed, bits)] @ hadamard() * (norms.astype(np.float64) / D)[..., None]


def attend(q, k, v, seen, scale, k_err, v_err):
    """softmax(scale q k^T) v over the first `seen` tokens for q [group, 256]; with it a bound on the 2-norm of the error
    of a kernel that carries key j with a relative error k_err[j] in every product q_d k_d, value j with v_err[j], and
    rounds the result to bf16."""
    k, v = k[:seen], v[:seen]
    s = scale * (q @ k.T)
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    o = p @ v
    # a score's error: its products' relative errors and 256 fp32 sums; as a relative error of p after normalising, twice
    ds = abs(scale) * np.linalg.norm(q, axis=-1)[:, None] * np.linalg.norm(k, axis=-1) * (k_err[:seen] + 2.0 ** -15)
    size = (p * np.linalg.norm(v, axis=-1)).sum(-1)
    # exp and the sum of up to 2^17 probabilities in fp32 with a running rescale: 2^-14 together
    off = 2 * ds.max(-1) + 2.0 ** -14
    bound = (np.expm1(off) * size + (p * v_err[:seen] * np.linalg.norm(v, axis=-1)).sum(-1)
             + 2.0 ** -8 * np.linalg.norm(o, axis=-1))
    return o, bound


# Relative errors of the operands.  Encoded tokens: q's rotation and the
# centroids are rounded to fp16 (2^-11 each), the norm is exact; p times the
# norm is rounded to fp16 (2^-11) or to a subnormal no coarser than that at the
# sizes tested, the centroid again 2^-11.  bf16 tokens: products are exact, p
# is rounded to bf16 (2^-8).
K_ERR = {True: 2 * 2.0 ** -11, False: 0.0}
V_ERR = {True: 2 * 2.0 ** -11, False: 2.0 ** -8}


def check_attention(out, q, keys, values, enc, base, kv_heads, scale=1 / 16):
    """out, q [rows, q_heads, 256] of one request in 64 bits; keys, values [kv_heads, tokens, 256], the first `enc` of
    them decoded from pages; row i sees the first base + i + 1."""
    rows, hq, _ = q.shape
    g = hq // kv_heads
    is_enc = np.arange(keys.shape[1]) < enc
    ke, ve = np.where(is_enc, K_ERR[True], K_ERR[False]), np.where(is_enc, V_ERR[True], V_ERR[False])
    worst = 0.0
    for i in range(rows):
        for h in range(kv_heads):
            o, bound = attend(q[i, h * g:(h + 1) * g], keys[h], values[h], base + i + 1, scale, ke, ve)
            err = np.linalg.norm(out[i, h * g:(h + 1) * g] - o, axis=-1)
            ok = err <= bound
            assert np.all(ok), f"row {i} kv head {h}: error {err[~ok][:4]}, bound {bound[~ok][:4]}"
            worst = max(worst, float((err / np.maximum(bound, 1e-300)).max()))
    assert math.isfinite(worst)
    return worst
