"""Cases of the paged KV-cache operators: what they compute, on what, and what it costs.

Four operators make one serving step over a paged cache of HLWQ codes:

* ``plan``   block tables, slot maps and positions from the requests' lengths;
* ``append`` a step's new keys and values into the window, the tokens they push out encoded into pages;
* ``attn``   attention of the step's new tokens over pages, window and themselves;
* ``prompt`` causal attention over whole prompts, packed one after the other.

``run`` computes them with elementary torch operations, or, where ``own`` is true, through the package.
"""
import math

import torch

own = False

D = 256  # head_dim of the KV path

# The codebooks of the KV path (Lloyd-Max for N(0, 1)) as the fp32 values the
# library documents, and the fp32 thresholds between their cells.
CENTROIDS = {
    3: (-2.1519455909729004, -1.3439092636108398, -0.7560052871704102, -0.2450941801071167,
        0.2450941801071167, 0.7560052871704102, 1.3439092636108398, 2.1519455909729004),
    2: (-1.5104175806045532, -0.4527800381183624, 0.4527800381183624, 1.5104175806045532),
}
THRESHOLDS = {
    3: (-1.7479274272918701, -1.049957275390625, -0.5005497336387634, 0.0,
        0.5005497336387634, 1.049957275390625, 1.7479274272918701),
    2: (-0.9815988540649414, 0.0, 0.9815987944602966),
}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 running requests: tables and slots for 64 rows
        dict(name="plan_decode_64", op="plan", requests=64, ctx_lo=1, ctx_hi=32767, new_lo=1, new_hi=1, pad=0, page=64,
             residual=128, reset_every=0),
        # a continuous-batching step: 1000 slots, decodes and chunks mixed, every 9th slot given up, padded rows
        dict(name="plan_mixed_1000", op="plan", requests=1000, ctx_lo=0, ctx_hi=32768, new_lo=0, new_hi=77, pad=1003,
             page=64, residual=128, reset_every=9),
        # the cache update of a decode step, 32 requests
        dict(name="append_decode_32_q3", op="append", requests=32, kv_heads=4, bits=3, ctx_lo=3, ctx_hi=32767, new_lo=1,
             new_hi=1, pad=0, page=64, residual=128, ring=144),
        # chunks of up to 128 tokens of 6 requests, 2-bit cache, K and V read out of one fused projection
        dict(name="append_chunk_6_q2", op="append", requests=6, kv_heads=2, bits=2, ctx_lo=90, ctx_hi=9001, new_lo=17,
             new_hi=128, pad=5, page=16, residual=128, ring=256),
        # a long prompt into the cache
        dict(name="append_prompt_16383_q3", op="append", requests=1, kv_heads=4, bits=3, ctx_lo=0, ctx_hi=0, new_lo=16383,
             new_hi=16383, pad=0, page=64, residual=128, ring=128),
        # one token of a short chat
        dict(name="attn_decode_1x500_q3", op="attn", requests=1, q_heads=24, kv_heads=4, bits=3, ctx_lo=500, ctx_hi=500,
             new_lo=1, new_hi=1, pad=0, page=64, residual=128, ring=128),
        # one token over the whole benchmark cache
        dict(name="attn_decode_1x32767_q3", op="attn", requests=1, q_heads=24, kv_heads=4, bits=3, ctx_lo=32767,
             ctx_hi=32767, new_lo=1, new_hi=1, pad=0, page=64, residual=128, ring=128),
        # a decode batch of requests of very different lengths, 2-bit cache
        dict(name="attn_decode_48_ragged_q2", op="attn", requests=48, q_heads=16, kv_heads=2, bits=2, ctx_lo=5,
             ctx_hi=16385, new_lo=1, new_hi=1, pad=0, page=64, residual=128, ring=128),
        # a chunk of a long prompt over what is cached of it
        dict(name="attn_chunk_1024_over_16000_q3", op="attn", requests=1, q_heads=24, kv_heads=4, bits=3, ctx_lo=16000,
             ctx_hi=16000, new_lo=1024, new_hi=1024, pad=0, page=64, residual=128, ring=128),
        # one short prompt of odd length
        dict(name="prompt_1x517", op="prompt", sequences=1, q_heads=24, kv_heads=4, len_lo=517, len_hi=517, pad=0),
        # a packed batch of prompts from one token to a few thousand
        dict(name="prompt_packed_9", op="prompt", sequences=9, q_heads=16, kv_heads=2, len_lo=1, len_hi=2500, pad=11),
        # one long prompt
        dict(name="prompt_1x16384", op="prompt", sequences=1, q_heads=24, kv_heads=4, len_lo=16384, len_hi=16384, pad=0),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)) - 1e-9)))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attn", "attn", "attn", "prompt", "prompt"])
    page = rng.choice([16, 32, 64, 128])
    residual = rng.choice([128, 128, 128, 64, 0, 37])
    q_heads, kv_heads = rng.choice([(24, 4), (16, 2), (8, 8), (8, 1), (12, 4), (20, 4)])
    bits = rng.choice([3, 2])
    if op == "plan":
        hi = _log(rng, 200, 32768)
        return dict(op=op, requests=_log(rng, 1, 900), ctx_lo=_log(rng, 1, 200) - 1, ctx_hi=hi, new_lo=rng.randint(0, 1),
                    new_hi=_log(rng, 1, 70), pad=rng.choice([0, 1, 29]), page=page, residual=residual,
                    reset_every=rng.choice([0, 2, 7]))
    if op == "append":
        if rng.random() < 0.5:  # steps over a filled cache
            new = _log(rng, 1, 100)
            return dict(op=op, requests=_log(rng, 1, 32), kv_heads=kv_heads, bits=bits, ctx_lo=_log(rng, 1, 300) - 1,
                        ctx_hi=_log(rng, 300, 9000), new_lo=rng.randint(0, 1) if new == 1 else rng.randint(0, new), new_hi=new,
                        pad=rng.choice([0, 3]), page=page, residual=residual, ring=residual + new + rng.randint(0, 40))
        requests = _log(rng, 1, 8)  # whole prompts
        new = _log(rng, 9, 12000 // requests)
        return dict(op=op, requests=requests, kv_heads=kv_heads, bits=bits, ctx_lo=0, ctx_hi=0, new_lo=_log(rng, 1, new),
                    new_hi=new, pad=rng.choice([0, 3]), page=page, residual=residual, ring=residual)
    if op == "attn":
        if rng.random() < 0.6:  # decode steps, a few drafted tokens among them
            requests = _log(rng, 1, 64)
            new = rng.choice([1, 1, 1, 2, 4, 5])
            hi = _log(rng, 200, min(32768, 600000 // requests))
        else:  # chunks, mixed with shorter ones
            requests = _log(rng, 1, 4)
            new = _log(rng, 6, 900 // requests)
            hi = _log(rng, 200, 15000 // requests)
        return dict(op=op, requests=requests, q_heads=q_heads, kv_heads=kv_heads, bits=bits, ctx_lo=rng.randint(0, hi),
                    ctx_hi=hi, new_lo=rng.randint(1, new), new_hi=new, pad=rng.choice([0, 0, 3]), page=page,
                    residual=residual, ring=residual + rng.choice([0, 0, 16]))
    sequences = _log(rng, 1, 10)
    hi = _log(rng, 2, 9000 // sequences)
    return dict(op=op, sequences=sequences, q_heads=q_heads, kv_heads=kv_heads, len_lo=_log(rng, 1, hi), len_hi=hi,
                pad=rng.choice([0, 0, 7]))


def _spread(lo, hi, count, salt):
    """`count` lengths of [lo, hi] in a fixed shuffled order, both ends among them."""
    if count == 1:
        return [hi]
    step = next(s for s in (7919, 104729, 1299709) if math.gcd(s, count) == 1)
    return [lo + (((i + salt) * step) % count) * (hi - lo) // (count - 1) for i in range(count)]


def _lengths(case):
    """(tokens held, new tokens, slots given up) of each request of a cache case."""
    n = case["requests"]
    ctx, new = _spread(case["ctx_lo"], case["ctx_hi"], n, 0), _spread(case["new_lo"], case["new_hi"], n, 3)
    every = case.get("reset_every", 0)
    gone = [bool(every) and i % every == every - 1 for i in range(n)]
    # a slot that is given up starts with what fits its window, so that the step can be planned again
    new = [min(x, case["residual"]) if g else x for x, g in zip(new, gone)]
    return ctx, new, gone


def _ceil(a, b):
    return -(-a // b)


def _encoded(tokens, residual):
    return max(tokens - residual, 0)


def work(case):
    if case["op"] == "prompt":
        lens = _spread(case["len_lo"], case["len_hi"], case["sequences"], 0)
        hq, hk = case["q_heads"], case["kv_heads"]
        return {"bytes": sum(lens) * (2 * hq + 2 * hk) * D * 2 + 4 * (len(lens) + 1),
                "flops": sum(4 * D * hq * (n * (n + 1) // 2) for n in lens)}
    ctx, new, gone = _lengths(case)
    res, page = case["residual"], case["page"]
    rows = sum(new) + case["pad"]
    if case["op"] == "plan":
        pages = 0
        for t, n, g in zip(ctx, new, gone):
            held = 0 if g else t
            if g:
                pages += 2 * _ceil(_encoded(t, res), page)  # read from the table, pushed
            pages += 2 * (_ceil(_encoded(held + n, res), page) - _ceil(_encoded(held, res), page))
        # slots need the page of each row that pushes a token out
        return {"bytes": 4 * (2 * len(ctx)) + len(ctx) + 4 * (2 * len(ctx) + 3) + 12 * rows + 4 * pages, "flops": 8 * rows}
    hk, vec = case["kv_heads"], 32 * case["bits"] + 2
    if case["op"] == "append":
        total = 0
        for t, n in zip(ctx, new):
            leave = _encoded(t + n, res) - _encoded(t, res)
            stay = min(n, res)
            from_ring = max(0, min(t, t + n - res) - max(t - res, 0))
            # every new token and every leaving ring token read once; codes, norm or ring slot written once
            total += n * 512 + from_ring * 512 + leave * vec + stay * 512
        return {"bytes": 2 * hk * total + 8 * rows, "flops": 2 * hk * sum(new) * D * 20}
    hq = case["q_heads"]
    nbytes = flops = 0
    for t, n in zip(ctx, new):
        e = _encoded(t, res)
        nbytes += 2 * hk * (e * vec + (t - e + n) * 512) + 2 * n * hq * 512 + 4 * _ceil(e, page)
        flops += 4 * D * hq * (n * t + n * (n + 1) // 2)
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _codes(g, shape, bits):
    """Packed codes of rotated unit-variance values, as the quantizer finds them."""
    z = torch.randn(*shape, D, device="cuda", generator=g)
    c = torch.bucketize(z, torch.tensor(THRESHOLDS[bits], device="cuda")).to(torch.int32)
    return _pack(c, bits)


def _pack(c, bits):
    """Codes [.., 256] to bytes [.., 32 * bits], 8 codes to `bits` bytes, first code in the lowest bits."""
    c = c.view(*c.shape[:-1], D // 8, 8)
    word = (c << (bits * torch.arange(8, device=c.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    byte = (word[..., None] >> (8 * torch.arange(bits, device=c.device, dtype=torch.int32))) & 255
    return byte.to(torch.uint8).flatten(-2)


def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prefix(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "prompt":
        lens = _spread(case["len_lo"], case["len_hi"], case["sequences"], 0)
        rows, hq, hk = sum(lens) + case["pad"], case["q_heads"], case["kv_heads"]
        qkv = _normal(g, rows, hq + 2 * hk, D)  # one projection's output, sliced
        qkv[:, :hq] *= 2
        return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], cu=_ints(_prefix(lens)),
                    longest=max(lens), out=torch.zeros(rows, hq, D, dtype=torch.bfloat16, device="cuda"))
    ctx, new, gone = _lengths(case)
    res, page, n = case["residual"], case["page"], case["requests"]
    rows = sum(new) + case["pad"]
    held = [0 if x else t for t, x in zip(ctx, gone)]
    before = [_ceil(_encoded(t, res), page) for t in ctx]
    after = [_ceil(_encoded(t + m, res), page) for t, m in zip(held, new)]
    width = max(max(before), max(after), 1) + 1
    pool = sum(before) + sum(max(a - b, 0) for a, b in zip(after, [0 if x else b for b, x in zip(before, gone)])) + 3
    ids = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    # the pages of the tokens held, then the stack of free ones
    used = _ints(before)
    first = torch.cumsum(used, 0) - used
    at = torch.arange(width, device="cuda")
    table = torch.where(at < used[:, None], ids[(first[:, None] + at).clamp(max=pool - 1)], -1).to(torch.int32)
    state = dict(case=case, rows=rows, table=table)
    if case["op"] == "plan":
        free = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
        free[:pool - sum(before)] = ids[sum(before):]
        state.update(tokens=_ints(ctx), new=_ints(new), reset=torch.tensor(gone, device="cuda").to(torch.uint8), free=free,
                     n_free=_ints([pool - sum(before)]))
        return state
    hk, bits, ring = case["kv_heads"], case["bits"], case["ring"]
    # what a plan of this step has given: prefix, lengths, and for the append its pages and slots
    cu = _prefix(new)
    lens = _ints([t + m for t, m in zip(ctx, new)])
    state.update(cu=_ints(cu), lens=lens)
    hq = case.get("q_heads", 0)
    qkv = _normal(g, rows, hq + 2 * hk, D)
    qkv[:, :hq] *= 2
    state.update(q=qkv[:, :hq], k_new=qkv[:, hq:hq + hk], v_new=qkv[:, hq + hk:])
    # slots of the pool that hold no token hold what an earlier request left, or nothing: NaN norms
    for x in "kv":
        state[x + "_packed"] = _codes(g, (pool, hk, page), bits)
        norms = torch.randn(pool, hk, page, device="cuda", generator=g).mul_(0.7).add_(16).to(torch.float16)
        live = torch.zeros(pool, page, dtype=torch.bool, device="cuda")
        enc = _ints([_encoded(t, res) for t in ctx])
        tok = at[:, None] * page + torch.arange(page, device="cuda")
        live[table.clamp(min=0)[at < used[:, None]].long()] = (tok[None] < enc[:, None, None])[at < used[:, None]]
        state[x + "_norms"] = torch.where(live[:, None, :], norms, float("nan")).to(torch.float16)
        state[x + "_window"] = _normal(g, n, hk, ring, D)
    if case["op"] == "append":
        have = _ints(after)
        grown = (at >= used[:, None]) & (at < have[:, None])
        table[grown] = ids[sum(before):sum(before) + int(grown.sum())]
        req = torch.repeat_interleave(torch.arange(n, device="cuda"), _ints(new))
        pos = torch.arange(cu[-1], device="cuda") - state["cu"][req] + _ints(ctx)[req]
        out = (pos - res).clamp(min=0)
        slot = torch.where(pos >= res, table[req, out // page] * page + out % page, -1).to(torch.int32)
        none = torch.full((case["pad"],), -1, dtype=torch.int32, device="cuda")
        state.update(row_request=torch.cat([req.to(torch.int32), none]), slots=torch.cat([slot, none]))
        return state
    state.update(out=torch.zeros(rows, hq, D, dtype=torch.bfloat16, device="cuda"),
                 most_held=max(ctx), most_new=max(new))
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"plan": _plan, "append": _append, "attn": _attn, "prompt": _prompt}[op](s)


def _own(s, op):
    import weight_quantization_amd as wq
    c = s["case"]
    if op == "plan":
        p = wq.hlwq_kv_page_plan(s["tokens"], s["new"], s["free"], s["n_free"], s["table"], s["rows"], page_size=c["page"],
                                 n_residual=c["residual"], reset=s["reset"])
        return dict(cu=p.cu_new, lens=p.lens, row_request=p.row_request, positions=p.positions, slots=p.slots,
                    n_free=p.n_free, status=p.status, free=s["free"], table=s["table"])
    if op == "append":
        wq.hlwq_kv_paged_append(s["k_new"], s["v_new"], s["cu"], s["lens"], s["row_request"], s["slots"], s["k_packed"],
                                s["k_norms"], s["v_packed"], s["v_norms"], s["k_window"], s["v_window"],
                                n_residual=c["residual"], bits=c["bits"])
        return {x + y: s[x + y] for x in "kv" for y in ("_packed", "_norms", "_window")}
    if op == "attn":
        return wq.hlwq_kv_paged_attention(s["q"], s["k_new"], s["v_new"], s["cu"], s["lens"], s["table"], s["k_packed"],
                                          s["k_norms"], s["v_packed"], s["v_norms"], s["k_window"], s["v_window"],
                                          n_residual=c["residual"], bits=c["bits"], out=s["out"])
    return wq.hlwq_prompt_attention(s["q"], s["k"], s["v"], s["cu"], out=s["out"])


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plan(s):
    c, dev = s["case"], "cuda"
    page, res, rows = c["page"], c["residual"], s["rows"]
    tokens, new, table, free = s["tokens"].long(), s["new"].long(), s["table"], s["free"]
    gone = s["reset"] != 0
    held = torch.where(gone, 0, tokens)
    lens = held + new
    zero = torch.zeros(1, dtype=torch.long, device=dev)
    cu = torch.cat([zero, torch.cumsum(new, 0)])
    at = torch.arange(table.shape[1], device=dev)

    def pages(t):
        return ((t - res).clamp(min=0) + page - 1) // page

    # give back the pages of the slots that end, in order
    back = gone[:, None] & (at < pages(tokens)[:, None])
    n_back, n_free = back.sum(), s["n_free"].long()
    order = torch.cumsum(back.flatten(), 0).view_as(back) - 1
    free[(n_free + order)[back]] = table[back]
    # take the new ones off the top
    had, want = pages(held), pages(lens)
    need = want - had
    first = torch.cumsum(need, 0) - need
    top = n_free + n_back
    grown = (at >= had[:, None]) & (at < want[:, None])
    take = (top - 1 - (first - had)[:, None] - at).clamp(0, free.shape[0] - 1)
    table.copy_(torch.where(grown, free[take], table))
    # rows
    i = torch.arange(rows, device=dev)
    req = torch.searchsorted(cu[1:], i, right=True)
    live = i < cu[-1]
    r = req.clamp(max=c["requests"] - 1)
    pos = i - cu[r] + held[r]
    old = (pos - res).clamp(min=0)
    slot = torch.where(live & (pos >= res), table[r, (old // page).clamp(max=table.shape[1] - 1)] * page + old % page, -1)
    i32 = torch.int32
    return dict(cu=cu.to(i32), lens=lens.to(i32), row_request=torch.where(live, req, -1).to(i32),
                positions=torch.where(live, pos, -1).to(i32), slots=slot.to(i32), n_free=(top - need.sum()).to(i32),
                status=torch.zeros(1, dtype=i32, device=dev), free=free, table=table)


def _tree(x):
    """Sum over the last axis, adjacent pairs first, one fp32 rounding a sum (squares of bf16 are exact)."""
    a = x[..., 0::2] + x[..., 1::2]
    a = a[..., 0::2] + a[..., 1::2]
    a = a[..., 0::2] + a[..., 1::2]
    a = a[..., 0::2] + a[..., 1::2]
    a = a[..., 0::2] + a[..., 1::2]
    a = a[..., 0::2] + a[..., 1::2]
    a = a[..., 0::2] + a[..., 1::2]
    a = a[..., 0::2] + a[..., 1::2]
    return a[..., 0]


def _butterfly(x, h):
    x = x.view(*x.shape[:-1], D // (2 * h), 2, h)
    a, b = x[..., 0, :], x[..., 1, :]
    return torch.stack((a + b, a - b), -2).flatten(-3)


def _encode(x, bits):
    """(packed codes, fp16 norms) of bf16 vectors [.., 256], in the fixed fp32 order of the KV quantizer."""
    x = x.float()
    n = _tree(x * x).double().sqrt().float()  # a 64-bit root rounded to 32 bits is the correctly rounded root
    r = torch.where(n >= torch.finfo(torch.float32).tiny, (1.0 / n.double()).float(), 0.0)
    y = _butterfly(_butterfly(_butterfly(_butterfly(x, 1), 2), 4), 8)
    y = _butterfly(_butterfly(_butterfly(_butterfly(y, 16), 32), 64), 128) * r[..., None]
    code = (y[..., None] > torch.tensor(THRESHOLDS[bits], device=y.device)).sum(-1, dtype=torch.int32)
    return _pack(code, bits), n.to(torch.float16)


def _append(s):
    c = s["case"]
    res, ring, page, hk = c["residual"], c["ring"], c["page"], c["kv_heads"]
    live = s["row_request"] >= 0
    i = torch.nonzero(live)[:, 0]
    req = s["row_request"][i].long()
    cu, lens = s["cu"].long(), s["lens"].long()
    held = lens - (cu[1:] - cu[:-1])
    pos = i - cu[req] + held[req]
    old = pos - res
    out = {}
    leave = s["slots"][i] >= 0
    slot = s["slots"][i][leave].long()
    stay = pos >= lens[req] - res
    for x in ("k", "v"):
        window, packed, norms, new = s[x + "_window"], s[x + "_packed"], s[x + "_norms"], s[x + "_new"]
        row, t, b = i[leave], old[leave], req[leave]
        ringed = window[b, :, (t % max(ring, 1))] if ring else new[row]
        source = torch.where((t < held[b])[:, None, None], ringed, new[(row - res).clamp(min=0)])
        codes, n16 = _encode(source, c["bits"])
        packed[slot // page, :, slot % page] = codes
        norms[slot // page, :, slot % page] = n16
        if ring:
            window[req[stay], :, pos[stay] % ring] = new[i[stay]]
        out.update({x + "_packed": packed, x + "_norms": norms, x + "_window": window})
    return out


def _hadamard(dtype):
    i = torch.arange(D, device="cuda")
    bits = i[:, None] & i[None, :]
    odd = sum((bits >> k) & 1 for k in range(8)) & 1
    return (1 - 2 * odd).to(dtype)


def _values(packed, bits):
    """Centroids [.., 256] of packed codes."""
    word = (packed.view(*packed.shape[:-1], D // 8, bits).to(torch.int32)
            << (8 * torch.arange(bits, device=packed.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    code = (word[..., None] >> (bits * torch.arange(8, device=packed.device, dtype=torch.int32))) & ((1 << bits) - 1)
    return torch.tensor(CENTROIDS[bits], device=packed.device)[code.flatten(-2)]


def _cached(s, x, enc, most):
    """The keys or values of every request as one padded fp32 tensor [requests, kv_heads, tokens, 256]."""
    c = s["case"]
    page, ring, res, bits, n = c["page"], c["ring"], c["residual"], c["bits"], c["requests"]
    cu, lens = s["cu"].long(), s["lens"].long()
    held = lens - (cu[1:] - cu[:-1])
    t = torch.arange(most, device="cuda")
    pages = s["table"][:, :max(1, _ceil(_encoded(s["most_held"], res), page))].clamp(min=0).long()
    packed, norms = s[x + "_packed"][pages], s[x + "_norms"][pages]  # [n, pages, heads, page, ..]
    old = _values(packed, bits) @ _hadamard(torch.float32) * (norms.float() / D)[..., None]
    old = old.permute(0, 2, 1, 3, 4).flatten(2, 3)
    live = t[:old.shape[2]] < enc[:, None]
    old = torch.where(live[:, None, :, None], old[:, :, :most], 0.0)
    full = torch.zeros(n, c["kv_heads"], most, D, device="cuda")
    full[:, :, :old.shape[2]] = old
    r = torch.arange(n, device="cuda")[:, None]
    if ring:
        w = (t >= enc[:, None]) & (t < held[:, None])
        b, tt = torch.nonzero(w, as_tuple=True)
        full[b, :, tt] = s[x + "_window"][b, :, tt % ring].float()
    w = (t >= held[:, None]) & (t < lens[:, None])
    b, tt = torch.nonzero(w, as_tuple=True)
    full[b, :, tt] = s[x + "_new"][cu[b] + tt - held[b]].float()
    return full


def _softmax_out(q, k, v, seen):
    """softmax(q k^T / 16 where seen) v, all fp32; rows that see nothing give 0."""
    score = q.matmul(k.transpose(-1, -2)).mul_(1 / 16).masked_fill_(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(torch.isfinite(top), top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    return p.matmul(v) / torch.where(total > 0, total, 1.0)


def _attn(s):
    c = s["case"]
    hk, n = c["kv_heads"], c["requests"]
    group = c["q_heads"] // hk
    cu, lens = s["cu"].long(), s["lens"].long()
    count = cu[1:] - cu[:-1]
    held = lens - count
    enc = (held - c["residual"]).clamp(min=0)
    most = s["most_held"] + s["most_new"]
    k, v = _cached(s, "k", enc, most), _cached(s, "v", enc, most)
    i = torch.arange(s["most_new"], device="cuda")
    b, ii = torch.nonzero(i < count[:, None], as_tuple=True)
    q = torch.zeros(n, s["most_new"], hk, group, D, device="cuda")
    q[b, ii] = s["q"][cu[b] + ii].float().view(-1, hk, group, D)
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)  # [n, hk, new * group, D]
    seen = torch.arange(most, device="cuda") <= (held[:, None] + i)[..., None]
    seen = seen & (i < count[:, None])[..., None]
    seen = seen.repeat_interleave(group, 1)[:, None]
    o = _softmax_out(q, k, v, seen).view(n, hk, s["most_new"], group, D).permute(0, 2, 1, 3, 4)
    s["out"][cu[b] + ii] = o[b, ii].flatten(1, 2).to(torch.bfloat16)
    return s["out"]


def _prompt(s):
    c = s["case"]
    hk, n, most = c["kv_heads"], c["sequences"], s["longest"]
    group = c["q_heads"] // hk
    cu = s["cu"].long()
    i = torch.arange(most, device="cuda")
    b, ii = torch.nonzero(i < (cu[1:] - cu[:-1])[:, None], as_tuple=True)

    def padded(x):
        y = torch.zeros(n, most, x.shape[1], D, device="cuda")
        y[b, ii] = x[cu[b] + ii].float()
        return y

    q = padded(s["q"]).view(n, most, hk, group, D).permute(0, 2, 3, 1, 4)
    k, v = (padded(s[x]).permute(0, 2, 1, 3)[:, :, None].contiguous() for x in ("k", "v"))
    o = _softmax_out(q, k, v, i <= i[:, None]).permute(0, 3, 1, 2, 4)
    s["out"][cu[b] + ii] = o[b, ii].flatten(1, 2).to(torch.bfloat16)
    return s["out"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _attend64(q, k, v, base):
    """Row r of q [rows, group, 256] sees the first base + r + 1 of k, v [tokens, 256]."""
    score = torch.einsum("rgd,td->rgt", q, k) / math.sqrt(D)
    t = torch.arange(k.shape[0], device=k.device)
    r = torch.arange(q.shape[0], device=k.device)
    score = score.masked_fill((t > base + r[:, None])[:, None], -math.inf)
    return torch.softmax(score, -1) @ v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None
    if op == "prompt":
        cu = s["cu"].tolist()
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        group = case["q_heads"] // case["kv_heads"]
        for a, b in zip(cu, cu[1:]):
            for h in range(case["kv_heads"]):
                k, v = s["k"][a:b, h].double(), s["v"][a:b, h].double()
                for r in range(a, b, 2048):
                    e = min(b, r + 2048)
                    hs = slice(h * group, (h + 1) * group)
                    out[r:e, hs] = _attend64(s["q"][r:e, hs].double(), k[:e - a], v[:e - a], r - a)
        return out
    ctx, new, _ = _lengths(case)
    cu, res, ring, page, bits = s["cu"].tolist(), case["residual"], case["ring"], case["page"], case["bits"]
    if op == "append":
        out = {}
        for x in "kv":
            norms, window = s[x + "_norms"].double(), s[x + "_window"].double()
            for r, (t, n) in enumerate(zip(ctx, new)):
                rows = s[x + "_new"][cu[r]:cu[r] + n].double()
                old = torch.arange(max(t - res, 0), max(t + n - res, 0), device="cuda")
                if old.numel():
                    held = window[r][:, old % ring].transpose(0, 1) if ring else rows[:0]
                    src = torch.where((old < t)[:, None, None], held, rows[(old - t).clamp(min=0)]) if ring else rows[old - t]
                    where = s["slots"][cu[r]:cu[r] + n].long()
                    where = where[where >= 0]
                    norms[where // page, :, where % page] = src.square().sum(-1).sqrt()
            for r, (t, n) in enumerate(zip(ctx, new)):
                rows = s[x + "_new"][cu[r]:cu[r] + n].double()
                at = torch.arange(max(t, t + n - res), t + n, device="cuda")
                if at.numel():
                    window[r][:, at % ring] = rows[at - t].transpose(0, 1)
            # the codes are defined by a fixed fp32 order and have no value in 64 bits
            out.update({x + "_packed": None, x + "_norms": norms, x + "_window": window})
        return out
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    group = case["q_heads"] // case["kv_heads"]
    book = torch.tensor(CENTROIDS[bits], dtype=torch.float64, device="cuda")
    had = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    for _ in range(8):
        had = torch.cat([torch.cat([had, had], 1), torch.cat([had, -had], 1)], 0)
    for r, (t, n) in enumerate(zip(ctx, new)):
        if n == 0:
            continue
        e = _encoded(t, res)
        ids = s["table"][r, :_ceil(e, page)].long()
        at = torch.arange(e, t, device="cuda")
        for h in range(case["kv_heads"]):
            both = []
            for x in "kv":
                raw = s[x + "_packed"][ids, h].reshape(-1, 32 * bits)[:e]
                bit = (raw[:, :, None] >> torch.arange(8, device="cuda")) & 1
                bit = bit.reshape(e, D, bits).long()
                code = (bit * (2 ** torch.arange(bits, device="cuda"))).sum(-1)
                norm = s[x + "_norms"][ids, h].reshape(-1)[:e].double()
                old = (book[code] / 16) @ (had / 16) * norm[:, None]
                near = s[x + "_window"][r, h][at % ring].double() if at.numel() else old[:0]
                both.append(torch.cat([old, near, s[x + "_new"][cu[r]:cu[r] + n, h].double()]))
            hs = slice(h * group, (h + 1) * group)
            for a in range(0, n, 512):
                z = min(n, a + 512)
                out[cu[r] + a:cu[r] + z, hs] = _attend64(s["q"][cu[r] + a:cu[r] + z, hs].double(), both[0][:t + z],
                                                         both[1][:t + z], t + a)
    return out
