"""Verification of drafted tokens step by step in Python, 64-bit sums, straight from the recursive rejection."""
import numpy as np


def verify(tokens, parents, cu, p, q, u, u_next, most=4096):
    """Returns n_kept, next_token, kept as hlwq_verify_drafts lays them out; p, q fp64 arrays [rows, vocab] or q None."""
    n, rows, vocab = len(cu) - 1, len(tokens), p.shape[1]
    n_kept, nxt, kept = np.zeros(n, np.int32), np.full(n, -1, np.int32), np.full(rows, -1, np.int32)
    for b in range(n):
        lo, hi = int(cu[b]), int(cu[b + 1])
        if lo == hi:
            continue
        cur, path = 0, [lo]
        base = p[lo]
        left, mass, taken = base.copy(), 1.0, 0.0  # (p - taken q)+ and the mass it is over
        for i in range(1, min(hi - lo, most)):
            x = int(tokens[lo + i])
            if parents[lo + i] != cur or not 0 <= x < vocab:
                continue
            qx = 1.0 if q is None else q[lo + cur, x]
            if float(u[lo + i]) * qx * mass < left[x]:
                cur = i
                path.append(lo + i)
                left, mass, taken = p[lo + i].copy(), 1.0, 0.0
            elif q is None:
                mass -= left[x]
                left[x] = 0
            else:
                taken += mass
                left = np.maximum(p[lo + cur] - taken * q[lo + cur], 0)
                mass = left.sum()
        if not left.sum() > 0:
            left = p[lo + cur].copy()
        n_kept[b] = len(path)
        kept[lo:lo + len(path)] = path
        if left.sum() > 0:
            upto = np.cumsum(left)
            at = int(np.searchsorted(upto, float(u_next[b]) * upto[-1], side="right"))
            nxt[b] = min(at, int(np.nonzero(left)[0][-1]))
    return n_kept, nxt, kept
