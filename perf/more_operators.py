"""Cases of the operators of a decode step of drafted tokens: what they compute, on what, and what it costs.

Three operators, beside the paged cache and the expert banks of HLWQ codes:

* ``tree``   attention of a tree of drafted tokens for each request, over pages, window and their own ancestors;
* ``moe``    a mixture-of-experts layer of a few tokens, router and experts, straight from the banks' codes;
* ``verify`` which drafted tokens stand against the target's probabilities, and the token that follows them.

``run`` computes them with elementary torch operations, or, where ``own`` is true, through the package.
"""
import math

import torch

own = False

D = 256    # head_dim of the KV path
B = 128    # weights to a block

# The codebooks (Lloyd-Max for N(0, 1)) as the fp32 values the library documents, and the thresholds
# between their cells, to draw codes with.
_POSITIVE = {
    5: (0.06588965654373169, 0.1980518251657486, 0.331378310918808, 0.4666995108127594, 0.6049336194992065,
        0.7471356987953186, 0.8945651054382324, 1.048783302307129, 1.2118043899536133, 1.3863403797149658,
        1.5762280225753784, 1.7872332334518433, 2.028728485107422, 2.317739486694336, 2.69111967086792, 3.260732412338257),
    3: (0.2450941801071167, 0.7560052871704102, 1.3439092636108398, 2.1519455909729004),
    2: (0.4527800381183624, 1.5104175806045532),
}
CENTROIDS = {b: tuple(-x for x in reversed(c)) + c for b, c in _POSITIVE.items()}
THRESHOLDS = {b: tuple((x + y) / 2 for x, y in zip(c, c[1:])) for b, c in CENTROIDS.items()}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a small tree behind a short chat
        dict(name="tree_1x9_over_500_q3", op="tree", requests=1, q_heads=24, kv_heads=4, bits=3, ctx_lo=500, ctx_hi=500,
             new_lo=9, new_hi=9, wide=4, pad=0, page=64, residual=128, ring=128),
        # a large tree over the whole benchmark cache
        dict(name="tree_1x64_over_32767_q3", op="tree", requests=1, q_heads=24, kv_heads=4, bits=3, ctx_lo=32767,
             ctx_hi=32767, new_lo=64, new_hi=64, wide=8, pad=0, page=64, residual=128, ring=128),
        # a batch of requests of very different lengths, trees of 1 to 33 nodes, 2-bit cache, padded rows
        dict(name="tree_24_ragged_q2", op="tree", requests=24, q_heads=16, kv_heads=2, bits=2, ctx_lo=5, ctx_hi=16385,
             new_lo=1, new_hi=33, wide=5, pad=3, page=64, residual=128, ring=128),
        # one token through the layer of 256 experts
        dict(name="moe_1_of_256x512_q5", op="moe", tokens=1, experts=256, hidden=2048, inner=512, top_k=8, bits=5, act="silu",
             renorm=True),
        # a few drafted tokens, 128 experts whose inner size ends in half a block
        dict(name="moe_5_of_128x704_q5", op="moe", tokens=5, experts=128, hidden=2816, inner=704, top_k=8, bits=5,
             act="gelu_tanh", renorm=True),
        # a decode batch of odd size, 3-bit bank, weights as the softmax leaves them
        dict(name="moe_17_of_256x512_q3", op="moe", tokens=17, experts=256, hidden=2048, inner=512, top_k=8, bits=3, act="silu",
             renorm=False),
        # a decode batch that touches most experts
        dict(name="moe_64_of_256x512_q5", op="moe", tokens=64, experts=256, hidden=2048, inner=512, top_k=8, bits=5, act="silu",
             renorm=True),
        # trees of several requests: every expert, several tokens each
        dict(name="moe_192_of_256x512_q5", op="moe", tokens=192, experts=256, hidden=2048, inner=512, top_k=8, bits=5,
             act="silu", renorm=True),
        # one request's chain of five drafts
        dict(name="verify_1_chain_5", op="verify", requests=1, new_lo=6, new_hi=6, wide=1, vocab=32000, dtype="float32",
             sampled=True, pad=0),
        # trees of sampled drafts, siblings among them
        dict(name="verify_48_trees", op="verify", requests=48, new_lo=1, new_hi=25, wide=4, vocab=131072, dtype="float32",
             sampled=True, pad=5),
        # chains of three drafts without a distribution of their own, 16-bit probabilities, odd vocabulary
        dict(name="verify_250_chains_bf16", op="verify", requests=250, new_lo=4, new_hi=4, wide=1, vocab=100003,
             dtype="bfloat16", sampled=False, pad=0),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)) - 1e-9)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "moe", "moe", "verify"])
    if op == "tree":
        q_heads, kv_heads = rng.choice([(24, 4), (16, 2), (8, 8), (8, 1), (12, 4), (20, 4)])
        residual = rng.choice([128, 128, 128, 64, 0, 37])
        requests = _log(rng, 1, 48)
        new = _log(rng, 1, min(64, 900 // requests))
        hi = _log(rng, 200, min(32768, 600000 // requests))
        return dict(op=op, requests=requests, q_heads=q_heads, kv_heads=kv_heads, bits=rng.choice([3, 2]),
                    ctx_lo=rng.randint(0, hi), ctx_hi=hi, new_lo=rng.randint(1, new), new_hi=new, wide=rng.randint(1, 9),
                    pad=rng.choice([0, 0, 3]), page=rng.choice([16, 32, 64, 128]), residual=residual,
                    ring=residual + rng.choice([0, 0, 16]))
    if op == "moe":
        experts, hidden, inner = rng.choice([(256, 2048, 512), (128, 2816, 704), (64, 1000, 200), (32, 5120, 1000),
                                             (8, 4096, 1408)])
        return dict(op=op, tokens=_log(rng, 1, 100), experts=experts, hidden=hidden, inner=inner,
                    top_k=rng.randint(1, min(8, experts // 2)), bits=rng.choice([5, 3]), act=rng.choice(["silu", "gelu_tanh"]),
                    renorm=rng.random() < 0.7)
    new = _log(rng, 1, 30)
    requests = _log(rng, 1, 600 // new)
    return dict(op=op, requests=requests, new_lo=rng.randint(1, new), new_hi=new, wide=rng.randint(1, 5),
                vocab=_log(rng, 500, 131072), dtype=rng.choice(["float32", "float32", "bfloat16", "float16"]),
                sampled=rng.random() < 0.6, pad=rng.choice([0, 0, 2]))


def _spread(lo, hi, count, salt):
    """`count` lengths of [lo, hi] in a fixed shuffled order, both ends among them."""
    if count == 1:
        return [hi]
    step = next(s for s in (7919, 104729, 1299709) if math.gcd(s, count) == 1)
    return [lo + (((i + salt) * step) % count) * (hi - lo) // (count - 1) for i in range(count)]


def _nodes(case):
    return _spread(case["new_lo"], case["new_hi"], case["requests"], 3)


def _held(case):
    return _spread(case["ctx_lo"], case["ctx_hi"], case["requests"], 0)


def _ceil(a, b):
    return -(-a // b)


def _encoded(tokens, residual):
    return max(tokens - residual, 0)


def work(case):
    if case["op"] == "tree":
        hq, hk, res, vec = case["q_heads"], case["kv_heads"], case["residual"], 32 * case["bits"] + 2
        nbytes = flops = 0
        for t, n in zip(_held(case), _nodes(case)):
            e = _encoded(t, res)
            nbytes += 2 * hk * (e * vec + (t - e + n) * 512) + 2 * n * hq * 512 + 4 * _ceil(e, case["page"]) + 4 * n
            flops += 4 * D * hq * n * (t + 1)  # a node sees at least itself
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "moe":
        t, e, h, i, k = (case[x] for x in ("tokens", "experts", "hidden", "inner", "top_k"))
        block = 16 * case["bits"] + 2
        touched = e * (1 - (1 - k / e) ** t)  # experts, if the router spreads evenly
        bank = 2 * i * _ceil(h, B) * block + h * _ceil(i, B) * block
        return {"bytes": int(touched * bank) + 2 * e * h + 4 * t * h + 8 * t * k, "flops": 6 * t * k * h * i + 2 * t * e * h}
    # a row of each distribution for every request, and what the walk looks up
    size = 4 if case["dtype"] == "float32" else 2
    rows = sum(_nodes(case))
    both = 2 if case["sampled"] else 1
    return {"bytes": case["requests"] * (case["vocab"] * size * both + 12) + rows * (16 + size * both),
            "flops": 4 * case["requests"] * case["vocab"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _codes(g, shape, n, bits):
    """Packed codes [.., n * bits / 8] of rotated unit-variance values, as the quantizer finds them."""
    z = torch.randn(*shape, n, device="cuda", generator=g)
    c = torch.bucketize(z, torch.tensor(THRESHOLDS[bits], device="cuda"))
    del z
    c = c.view(*shape, n // 8, 8)
    word = torch.zeros(*shape, n // 8, dtype=torch.int64, device="cuda")
    for i in range(8):
        word |= c[..., i] << (bits * i)
    return torch.stack([(word >> (8 * i)).to(torch.uint8) for i in range(bits)], -1).flatten(-2)


def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prefix(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


def _parents(case, g):
    """Trees of the requests' nodes: a node hangs on one of the `wide` before it; -1 for each first and for padding."""
    nodes = _nodes(case)
    at = torch.cat([torch.arange(n, device="cuda") for n in nodes] + [torch.zeros(case["pad"], device="cuda")]).long()
    back = (torch.rand(at.numel(), device="cuda", generator=g) * case["wide"]).long() + 1
    return torch.where(at > 0, (at - back).clamp(min=0), -1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"tree": _prepare_tree, "moe": _prepare_moe, "verify": _prepare_verify}[case["op"]](case, g)


def _prepare_tree(case, g):
    ctx, new, res, page, n = _held(case), _nodes(case), case["residual"], case["page"], case["requests"]
    rows, hk, hq, bits, ring = sum(new) + case["pad"], case["kv_heads"], case["q_heads"], case["bits"], case["ring"]
    used = [_ceil(_encoded(t, res), page) for t in ctx]
    width, pool = max(used) + 1, sum(used) + 3
    ids = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    have = _ints(used)
    at = torch.arange(width, device="cuda")
    first = torch.cumsum(have, 0) - have
    table = torch.where(at < have[:, None], ids[(first[:, None] + at).clamp(max=pool - 1)], -1).to(torch.int32)
    qkv = _normal(g, rows, hq + 2 * hk, D)  # one projection's output, sliced
    qkv[:, :hq] *= 2
    state = dict(case=case, table=table, cu=_ints(_prefix(new)), lens=_ints([t + m for t, m in zip(ctx, new)]),
                 parents=_parents(case, g), q=qkv[:, :hq], k_new=qkv[:, hq:hq + hk], v_new=qkv[:, hq + hk:],
                 out=torch.zeros(rows, hq, D, dtype=torch.bfloat16, device="cuda"))
    # slots of the pool that hold no token hold what an earlier request left, or nothing: NaN norms
    live = torch.zeros(pool, page, dtype=torch.bool, device="cuda")
    enc = _ints([_encoded(t, res) for t in ctx])
    tok = at[:, None] * page + torch.arange(page, device="cuda")
    mine = at < have[:, None]
    live[table[mine].long()] = (tok[None] < enc[:, None, None])[mine]
    for x in "kv":
        state[x + "_packed"] = _codes(g, (pool, hk, page), D, bits)
        norms = torch.randn(pool, hk, page, device="cuda", generator=g).mul_(0.7).add_(16)
        state[x + "_norms"] = torch.where(live[:, None, :], norms, float("nan")).to(torch.float16)
        state[x + "_window"] = _normal(g, n, hk, ring, D)
    return state


def _prepare_moe(case, g):
    t, e, h, i, bits = (case[x] for x in ("tokens", "experts", "hidden", "inner", "bits"))

    def bank(out, n_in):
        nb = _ceil(n_in, B)
        packed = torch.empty(e, out, nb, 16 * bits, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (out * nb * B))
        for a in range(0, e, step):
            packed[a:a + step] = _codes(g, (min(step, e - a), out, nb), B, bits)
        # norms of blocks of N(0, 0.02^2), an outlier twenty times as large in every eighth; the last block of a row may be short
        norms = torch.randn(e, out, nb, device="cuda", generator=g).mul_(0.0142).add_(0.226)
        norms = torch.where(torch.rand(e, out, nb, device="cuda", generator=g) < 0.125, (norms * norms + 0.15).sqrt(), norms)
        norms[..., -1] *= math.sqrt((n_in - (nb - 1) * B) / B)
        return packed, norms.to(torch.float16)

    x = torch.randn(t, h, device="cuda", generator=g)
    x[:, torch.randperm(h, device="cuda", generator=g)[:h // 100]] *= 8  # a few large channels
    gate_up, down = bank(2 * i, h), bank(h, i)
    return dict(case=case, x=x.to(torch.bfloat16), router=_normal(g, e, h, scale=1.5 / math.sqrt(h)), gate_up=gate_up, down=down,
                out=torch.zeros(t, h, dtype=torch.bfloat16, device="cuda"))


def _prepare_verify(case, g):
    n, vocab, nodes = case["requests"], case["vocab"], _nodes(case)
    rows = sum(nodes) + case["pad"]
    dtype = getattr(torch, case["dtype"])
    parents = _parents(case, g)
    cu = _ints(_prefix(nodes))
    start = torch.repeat_interleave(cu[:-1], cu[1:] - cu[:-1])
    source = torch.zeros(rows, dtype=torch.long, device="cuda")
    source[:start.numel()] = start + parents[:start.numel()].clamp(min=0)  # the row whose distribution a token came from
    target = torch.empty(rows, vocab, dtype=dtype, device="cuda")
    draft = torch.empty(rows, vocab, dtype=dtype, device="cuda")
    step = max(1, (1 << 26) // vocab)
    for a in range(0, rows, step):
        z = torch.randn(min(step, rows - a), vocab, device="cuda", generator=g) * 3
        target[a:a + step] = torch.softmax(z, -1).to(dtype)
        z += torch.randn(*z.shape, device="cuda", generator=g) * 0.7  # a smaller model of the same text
        draft[a:a + step] = torch.softmax(z, -1).to(dtype)
    tokens = torch.empty(rows, dtype=torch.int32, device="cuda")
    for a in range(0, rows, step):
        q = draft[source[a:a + step]].float()
        if case["sampled"]:
            tokens[a:a + step] = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32)
        else:  # the best tokens, one for each sibling
            best = torch.topk(q, 10, -1).indices
            pick = torch.arange(a, a + q.shape[0], device="cuda") % case["wide"]
            tokens[a:a + step] = best.gather(1, pick[:, None])[:, 0].to(torch.int32)
    return dict(case=case, tokens=tokens, parents=parents, cu=cu, target=target, draft=draft if case["sampled"] else None,
                u=torch.rand(rows, device="cuda", generator=g), u_next=torch.rand(n, device="cuda", generator=g),
                most=max(nodes))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"tree": _tree, "moe": _moe, "verify": _verify}[op](s)


def _own(s, op):
    import weight_quantization_amd as wq
    c = s["case"]
    if op == "tree":
        return wq.hlwq_kv_tree_attention(s["q"], s["k_new"], s["v_new"], s["parents"], s["cu"], s["lens"], s["table"],
                                         s["k_packed"], s["k_norms"], s["v_packed"], s["v_norms"], s["k_window"],
                                         s["v_window"], n_residual=c["residual"], bits=c["bits"], out=s["out"])
    if op == "moe":
        y = wq.hlwq_moe_layer(s["x"], s["router"], *s["gate_up"], *s["down"], top_k=c["top_k"], bits=c["bits"],
                              activation=c["act"], renormalize=c["renorm"], out=s["out"])
        return dict(out=y.out, experts=y.experts, weights=y.weights)
    v = wq.hlwq_verify_drafts(s["tokens"], s["parents"], s["cu"], s["target"], s["u"], s["u_next"], draft=s["draft"])
    return dict(n_kept=v.n_kept, next_token=v.next_token, kept=v.kept)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _hadamard(n, dtype):
    i = torch.arange(n, device="cuda")
    both = i[:, None] & i[None, :]
    odd = sum((both >> k) & 1 for k in range(n.bit_length() - 1)) & 1
    return (1 - 2 * odd).to(dtype)


def _values(packed, bits):
    """fp32 centroids [.., n] of packed codes [.., n * bits / 8]."""
    group = packed.view(*packed.shape[:-1], -1, bits).to(torch.int64)
    word = (group << (8 * torch.arange(bits, device="cuda"))).sum(-1)
    code = (word[..., None] >> (bits * torch.arange(8, device="cuda"))) & ((1 << bits) - 1)
    return torch.tensor(CENTROIDS[bits], device="cuda")[code.flatten(-2)]


def _cached(s, x, enc, most):
    """The keys or values of every request as one padded fp32 tensor [requests, kv_heads, tokens, 256]."""
    c = s["case"]
    ring, res, bits, n = c["ring"], c["residual"], c["bits"], c["requests"]
    cu, lens = s["cu"].long(), s["lens"].long()
    held = lens - (cu[1:] - cu[:-1])
    t = torch.arange(most, device="cuda")
    pages = s["table"][:, :max(1, _ceil(_encoded(c["ctx_hi"], res), c["page"]))].clamp(min=0).long()
    packed, norms = s[x + "_packed"][pages], s[x + "_norms"][pages]  # [n, pages, heads, page, ..]
    old = _values(packed, bits) @ _hadamard(D, torch.float32) * (norms.float() / D)[..., None]
    old = old.permute(0, 2, 1, 3, 4).flatten(2, 3)
    old = torch.where((t[:old.shape[2]] < enc[:, None])[:, None, :, None], old[:, :, :most], 0.0)
    full = torch.zeros(n, c["kv_heads"], most, D, device="cuda")
    full[:, :, :old.shape[2]] = old
    if ring:
        b, tt = torch.nonzero((t >= enc[:, None]) & (t < held[:, None]), as_tuple=True)
        full[b, :, tt] = s[x + "_window"][b, :, tt % ring].float()
    b, tt = torch.nonzero((t >= held[:, None]) & (t < lens[:, None]), as_tuple=True)
    full[b, :, tt] = s[x + "_new"][cu[b] + tt - held[b]].float()
    return full


def _tree(s):
    c = s["case"]
    hk, n, wide = c["kv_heads"], c["requests"], c["new_hi"]
    group = c["q_heads"] // hk
    cu, lens = s["cu"].long(), s["lens"].long()
    count = cu[1:] - cu[:-1]
    held = lens - count
    enc = (held - c["residual"]).clamp(min=0)
    most = c["ctx_hi"] + wide
    k, v = _cached(s, "k", enc, most), _cached(s, "v", enc, most)
    i = torch.arange(wide, device="cuda")
    live = i < count[:, None]
    row = torch.where(live, cu[:-1, None] + i, 0)
    # who sees whom within a tree: a node what its parent sees, and itself
    parent = torch.where(live, s["parents"][row].long(), -1)
    kin = torch.zeros(n, wide, wide, dtype=torch.bool, device="cuda")
    each = torch.arange(n, device="cuda")
    for j in range(wide):
        p = parent[:, j]
        kin[:, j] = kin[each, p.clamp(min=0)] & (p >= 0)[:, None]
        kin[:, j, j] = True
    t = torch.arange(most, device="cuda")
    own_at = (t - held[:, None]).clamp(0, wide - 1)  # [n, most]
    among = torch.gather(kin, 2, own_at[:, None, :].expand(n, wide, most))
    seen = (t < held[:, None])[:, None] | ((t < lens[:, None])[:, None] & among)
    seen = (seen & live[..., None]).repeat_interleave(group, 1)[:, None]
    q = torch.where(live[..., None, None], s["q"][row].float(), 0.0)
    q = q.view(n, wide, hk, group, D).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [n, hk, nodes * group, D]
    score = q.matmul(k.transpose(-1, -2).contiguous()).mul_(1 / 16).masked_fill_(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(torch.isfinite(top), top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.matmul(v) / torch.where(total > 0, total, 1.0)).view(n, hk, wide, group, D).permute(0, 2, 1, 3, 4)
    s["out"][row[live]] = o[live].flatten(1, 2).to(torch.bfloat16)
    return s["out"]


def _act(x, name):
    if name == "silu":
        return x / (1 + torch.exp(-x))
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))


def _weights(packed, norms, n_in, bits):
    """fp32 weights [.., out, in] of a bank's codes and norms."""
    w = _values(packed, bits) @ _hadamard(B, torch.float32) * (norms.float() / B)[..., None]
    return w.flatten(-2)[..., :n_in]


def _moe(s):
    c = s["case"]
    x, k, e, bits, hidden, inner = s["x"], c["top_k"], c["experts"], c["bits"], c["hidden"], c["inner"]
    logits = x.double() @ s["router"].double().T
    top, ids = torch.sort(logits, stable=True, dim=-1, descending=True)  # ties: the lowest index first
    top, ids = top[:, :k], ids[:, :k]
    high = top[:, :1]
    total = (torch.exp(top - high) if c["renorm"] else torch.exp(logits - high)).sum(-1, keepdim=True)
    weights = (torch.exp(top - high) / total).float()
    xf = x.float()
    pairs = ids.numel()
    step = max(1, (1 << 26) // (2 * inner * hidden))
    if pairs <= e:  # the chosen experts' weights, pair by pair
        flat, token = ids.flatten(), torch.arange(pairs, device="cuda") // k
        y = torch.empty(pairs, hidden, device="cuda")
        for a in range(0, pairs, step):
            f, at = flat[a:a + step], token[a:a + step]
            gu = torch.bmm(_weights(s["gate_up"][0][f], s["gate_up"][1][f], hidden, bits), xf[at][..., None])[..., 0]
            h = _act(gu[:, :inner], c["act"]) * gu[:, inner:]
            y[a:a + step] = torch.bmm(_weights(s["down"][0][f], s["down"][1][f], inner, bits), h[..., None])[..., 0]
        y = (y.view(*ids.shape, hidden) * weights[..., None]).sum(1)
    else:  # every expert for every token, most of them with weight 0
        gate = torch.zeros(x.shape[0], e, device="cuda").scatter_(1, ids, weights)
        y = torch.zeros(x.shape[0], hidden, device="cuda")
        for a in range(0, e, step):
            w = _weights(s["gate_up"][0][a:a + step], s["gate_up"][1][a:a + step], hidden, bits)
            gu = torch.matmul(w, xf.T.contiguous())  # [experts, 2 inner, tokens]
            h = _act(gu[:, :inner], c["act"]) * gu[:, inner:] * gate[:, a:a + step].T[:, None]
            w = _weights(s["down"][0][a:a + step], s["down"][1][a:a + step], inner, bits)
            y += torch.matmul(w, h).sum(0).T
    s["out"].copy_(y.to(torch.bfloat16))
    return dict(out=s["out"], experts=ids.to(torch.int32), weights=weights)


def _verify(s):
    c = s["case"]
    cu, parents, tokens = s["cu"].long(), s["parents"].long(), s["tokens"].long()
    p, q, vocab, n = s["target"], s["draft"], c["vocab"], c["requests"]
    start, count = cu[:-1], cu[1:] - cu[:-1]
    each = torch.arange(n, device="cuda")
    last = p.shape[0] - 1

    def rows(node):
        return (start + node).clamp(max=last)

    cur = torch.zeros(n, dtype=torch.long, device="cuda")
    mass = torch.ones(n, dtype=torch.float64, device="cuda")    # of the residual
    taken = torch.zeros(n, dtype=torch.float64, device="cuda")  # multiples of q taken off p
    gone = torch.zeros(n, vocab, dtype=torch.bool, device="cuda") if q is None else None
    n_kept = (count > 0).long()
    kept = torch.full((p.shape[0] + 1,), -1, dtype=torch.long, device="cuda")  # the last takes what is not kept
    kept[torch.where(count > 0, start, last + 1)] = start
    for i in range(1, s["most"]):
        node = torch.full_like(cur, i)
        r, at = rows(node), rows(cur)
        child = (i < count) & (parents[r] == cur)
        x = tokens[r]
        px = p[at, x].double()
        if q is None:
            qx = torch.ones_like(px)
            value = torch.where(gone[each, x], 0.0, px)
        else:
            qx = q[at, x].double()
            value = (px - taken * qx).clamp(min=0)
        yes = child & (s["u"][r].double() * qx * mass < value)
        no = child & ~yes
        if q is None:
            mass = torch.where(no, mass - value, mass)
            gone[each, x] |= no
            gone &= ~yes[:, None]
        else:
            taken = torch.where(no, taken + mass, taken)
            rest = (p[at].double() - taken[:, None] * q[at].double()).clamp_(min=0).sum(-1)
            mass = torch.where(no, rest, mass)
        cur = torch.where(yes, node, cur)
        mass, taken = torch.where(yes, 1.0, mass), torch.where(yes, 0.0, taken)
        kept[torch.where(yes, start + n_kept, last + 1)] = r
        n_kept = n_kept + yes
    rest = p[rows(cur)].double()
    if q is None:
        left = torch.where(gone, 0.0, rest)
    else:
        left = (rest - taken[:, None] * q[rows(cur)].double()).clamp_(min=0)
    left = torch.where((left.sum(-1) > 0)[:, None], left, rest)
    upto = torch.cumsum(left, -1)
    nxt = (upto <= (s["u_next"].double() * upto[:, -1])[:, None]).sum(-1)
    top = torch.where(left > 0, torch.arange(vocab, device="cuda"), -1).amax(-1)
    i32 = torch.int32
    return dict(n_kept=n_kept.to(i32), next_token=torch.where(count > 0, torch.minimum(nxt, top), -1).to(i32),
                kept=kept[:-1].to(i32))


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _sylvester(n):
    had = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    while had.shape[0] < n:
        had = torch.cat([torch.cat([had, had], 1), torch.cat([had, -had], 1)], 0)
    return had


def _decoded(raw, bits, n):
    """64-bit vectors [m, n] (before the norm) of packed codes [m, n * bits / 8]: bit by bit."""
    bit = (raw[:, :, None] >> torch.arange(8, device="cuda")) & 1
    code = (bit.reshape(raw.shape[0], n, bits).long() * (2 ** torch.arange(bits, device="cuda"))).sum(-1)
    book = torch.tensor(CENTROIDS[bits], dtype=torch.float64, device="cuda")
    return book[code] @ _sylvester(n) / n


def _exact_tree(case, s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    group = case["q_heads"] // case["kv_heads"]
    cu, parents, res, ring = s["cu"].tolist(), s["parents"].tolist(), case["residual"], case["ring"]
    for r, (t, n) in enumerate(zip(_held(case), _nodes(case))):
        e = _encoded(t, res)
        ids = s["table"][r, :_ceil(e, case["page"])].long()
        at = torch.arange(e, t, device="cuda")
        seen = torch.zeros(n, n, dtype=torch.bool)
        for j in range(n):
            a = j
            while a >= 0:
                seen[j, a] = True
                a = parents[cu[r] + a]
        seen = torch.cat([torch.ones(n, t, dtype=torch.bool), seen], 1).cuda()
        for h in range(case["kv_heads"]):
            both = []
            for x in "kv":
                raw = s[x + "_packed"][ids, h].reshape(-1, 32 * case["bits"])[:e]
                norm = s[x + "_norms"][ids, h].reshape(-1)[:e].double()
                near = s[x + "_window"][r, h][at % ring].double() if at.numel() else norm.new_zeros(0, D)
                both.append(torch.cat([_decoded(raw, case["bits"], D) * norm[:, None], near,
                                       s[x + "_new"][cu[r]:cu[r] + n, h].double()]))
            hs = slice(h * group, (h + 1) * group)
            q = s["q"][cu[r]:cu[r] + n, hs].double()
            score = (q.reshape(-1, D) @ both[0].T).view(n, group, t + n) / math.sqrt(D)
            score = score.masked_fill(~seen[:, None], -math.inf)
            out[cu[r]:cu[r] + n, hs] = (torch.softmax(score, -1).view(-1, t + n) @ both[1]).view(n, group, D)
    return out


def _exact_moe(case, s):
    x, k, inner, bits = s["x"].double(), case["top_k"], case["inner"], case["bits"]
    prob = torch.softmax(x @ s["router"].double().T, -1)
    top, ids = torch.topk(prob, k, -1)
    if case["renorm"]:
        top = top / top.sum(-1, keepdim=True)
    y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")

    def matrix(bank, e, n_in):
        packed, norms = bank
        w = _decoded(packed[e].reshape(-1, 16 * bits), bits, B) * norms[e].reshape(-1, 1).double()
        return w.view(packed.shape[1], -1)[:, :n_in]

    for e in torch.unique(ids).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = x[t] @ matrix(s["gate_up"], e, case["hidden"]).T
        gate, up = gu[:, :inner], gu[:, inner:]
        if case["act"] == "silu":
            gate = gate * torch.sigmoid(gate)
        else:
            gate = gate / 2 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)))
        y[t] += top[t, j][:, None] * ((gate * up) @ matrix(s["down"], e, inner).T)
    return dict(out=y, experts=None, weights=top)  # which experts: whole numbers


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers
    s = prepare(case, seed)
    return _exact_tree(case, s) if case["op"] == "tree" else _exact_moe(case, s)
