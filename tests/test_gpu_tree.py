"""GPU tests of the attention of trees of drafted tokens against the definition over the operands that the kernels document
(tests/attention_bound.py), and of a whole step of drafted tokens."""
import numpy as np
import pytest

import attention_bound as ab
import paged_ref as pr
import verify_ref as vr
from test_gpu_attention_exact import sides
from test_gpu_paged import Cache, D, bf16_bits, dev16, f64, i32, strided, wq  # noqa: F401
from test_gpu_verify import softmax, trees

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def way(parents, i):
    """Node i of a request and its ancestors, as the kernels read the parents, oldest first."""
    out = []
    while i >= 0:
        out.append(i)
        i = parents[i] if -1 <= parents[i] < i else -1
    return out[::-1]


def check_tree(got, q, keys, values, held, parents, nodes, scale=1 / 16):
    """got, q [nodes, q_heads, 256] of one request in 64 bits; keys, values: a Side a KV head, the window's tokens and
    then the step's; `nodes` of them are looked at."""
    g, worst = q.shape[1] // len(keys), 0.0
    for i in nodes:
        mine = way(parents, i)
        for h, (k, v) in enumerate(zip(keys, values)):
            near = held - len(k.norms)
            keep = np.concatenate([np.arange(near), near + np.array(mine, int)]).astype(int)
            own = [ab.Side(x.cent, x.norms, x.near[keep]) for x in (k, v)]
            heads = slice(h * g, (h + 1) * g)
            o, bound = ab.expect(q[i, heads], *own, np.full(g, held + len(mine)), scale)
            err = np.linalg.norm(got[i, heads] - o, axis=-1)
            assert np.all(err <= bound), (i, h, err, bound)
            worst = max(worst, float((err / np.maximum(bound, 1e-300)).max()))
    return worst


def tree_case(wq, seed, ctx, new, q_heads, kv_heads, bits=3, page=64, residual=128, ring=128, wide=3, scale=1 / 16, extra=0,
              pad=0, parents=None, sigma=1.0, width=None):
    rng = np.random.default_rng(seed)
    c = Cache(rng, ctx, kv_heads, bits, page, residual, ring, width=width)
    n = sum(new) + pad
    q, kv = bf16_bits(rng, n, q_heads, D, sigma=sigma), [bf16_bits(rng, n, kv_heads, D) for _ in range(2)]
    cu = np.concatenate([[0], np.cumsum(new)])
    parents = np.concatenate([trees(rng, new, wide), np.full(pad, 5, np.int32)]) if parents is None else np.asarray(parents, np.int32)
    make = (lambda x: strided(x, extra)) if extra else dev16
    out = torch.full((n, q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    wq.hlwq_kv_tree_attention(make(q), make(kv[0]), make(kv[1]), i32(parents), i32(cu), i32([t + m for t, m in zip(ctx, new)]),
                              i32(c.table), *c.tensors(), n_residual=residual, bits=bits, scale=scale, out=out)
    got, worst = out.cpu().double().numpy(), 0.0
    assert np.all(got[cu[-1]:] == 7)
    for b, (t, m) in enumerate(zip(ctx, new)):
        r = slice(cu[b], cu[b + 1])
        nodes = range(m) if m <= 24 else np.unique(np.concatenate([[0, m - 1, m - 2], rng.integers(0, m, 16)]))
        worst = max(worst, check_tree(got[r], f64(q[r]), *sides(c, b, t, [x[r] for x in kv]), t, parents[r], nodes, scale))
    print(f"largest error {worst:.3f} of its bound", flush=True)


@pytest.mark.parametrize("ctx,new", [
    ([0], [1]), ([0], [7]), ([1], [2]), ([128], [5]), ([129], [9]), ([500], [33]), ([2049], [4]), ([5000], [64]),
    ([0, 1, 15, 128, 129, 144, 145, 192, 193, 1000, 3000], [1, 2, 3, 4, 5, 6, 7, 8, 16, 17, 18]), ([1000, 30], [40, 0]),
    ([4000, 0, 999], [3, 1, 0]), ([96, 97, 127], [32, 31, 33]),
])
@pytest.mark.parametrize("q_heads,kv_heads,bits,page", [(24, 4, 3, 64), (6, 2, 2, 16)])
def test_lengths(wq, ctx, new, q_heads, kv_heads, bits, page):
    tree_case(wq, sum(ctx) + len(new), ctx, new, q_heads, kv_heads, bits, page)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (8, 8), (8, 1), (20, 4), (17, 1), (64, 2)])
@pytest.mark.parametrize("bits", [3, 2])
def test_heads(wq, q_heads, kv_heads, bits):
    tree_case(wq, q_heads, [333, 40], [9, 21], q_heads, kv_heads, bits, 32, wide=5)


@pytest.mark.parametrize("residual,ring", [(0, 0), (1, 1), (37, 37), (64, 100), (128, 1000)])
@pytest.mark.parametrize("bits,page,new", [(3, 16, [1, 5, 3]), (2, 256, [30, 10, 2])])
def test_windows(wq, residual, ring, bits, page, new):
    tree_case(wq, residual + page, [residual + 50, 700, 20], new, 6, 2, bits, page, residual, ring)


@pytest.mark.parametrize("extra,pad", [(0, 5), (8, 0), (40, 3)])
def test_strides_and_padding(wq, extra, pad):
    tree_case(wq, extra, [300, 3], [12, 7], 6, 2, extra=extra, pad=pad)


@pytest.mark.parametrize("scale,sigma", [(0.0, 1.0), (-1 / 16, 1.0), (1.0, 1.0), (1 / 16, 8.0)])
def test_scales(wq, scale, sigma):
    tree_case(wq, 3, [300], [12], 6, 2, scale=scale, sigma=sigma)


@pytest.mark.parametrize("wide", [1, 1000])
@pytest.mark.parametrize("new", [[300], [1100, 257]])
def test_large_trees(wq, new, wide):
    # chains, and stars
    tree_case(wq, wide, [200] * len(new), new, 2, 1, wide=wide)


def test_a_chain_is_what_paged_attention_gives(wq):
    rng = np.random.default_rng(2)
    c = Cache(rng, [400, 7], 2, 3, 64, 128, 128)
    q, kv = bf16_bits(rng, 10, 6, D), [bf16_bits(rng, 10, 2, D) for _ in range(2)]
    t = [dev16(q), dev16(kv[0]), dev16(kv[1])]
    rest = (i32([0, 4, 10]), i32([404, 13]), i32(c.table), *c.tensors())
    a = wq.hlwq_kv_paged_attention(*t, *rest)
    b = wq.hlwq_kv_tree_attention(*t, i32([-1, 0, 1, 2, -1, 0, 1, 2, 3, 4]), *rest)
    assert torch.equal(a, b)


def test_parents_out_of_range_count_as_none(wq):
    parents = [0, 0, 2 ** 31 - 1, -2 ** 31, 4, 3, -1, 9, 1]
    tree_case(wq, 5, [150], [9], 6, 2, parents=parents)


def test_nan_and_infinities_stay_with_the_rows_that_see_them(wq):
    rng = np.random.default_rng(6)
    for new in ([12, 3], [50, 21]):
        ctx, n = [300, 20], sum(new)
        c = Cache(rng, ctx, 2, 3, 64, 128, 128)
        q, kv = bf16_bits(rng, n, 4, D), [bf16_bits(rng, n, 2, D) for _ in range(2)]
        parents = trees(rng, new, 4)
        rest = (i32(parents), i32([0, new[0], n]), i32([t + m for t, m in zip(ctx, new)]), i32(c.table), *c.tensors())
        clean = wq.hlwq_kv_tree_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), *rest)
        ways = [way(parents[:new[0]], i) for i in range(new[0])]
        # the node of request 0 that holds it: of those with a sibling's side of the tree, the one with most below it
        bad = max(range(1, new[0]), key=lambda x: sum(x in w for w in ways) % (new[0] - 1))
        rows = [i for i in range(new[0]) if bad in ways[i]]
        assert 1 < len(rows) < new[0] - 1
        for i, what in ((0, 0x7FC0), (1, 0x7FC0), (1, 0x7F80), (1, 0xFF80)):
            dirty = [x.copy() for x in kv]
            dirty[i][bad, 1, 17] = what
            got = wq.hlwq_kv_tree_attention(dev16(q), dev16(dirty[0]), dev16(dirty[1]), *rest)
            hit = torch.zeros(n, 4, D, dtype=torch.bool, device="cuda")
            if i == 0:
                hit[rows, 2:] = True
            else:
                hit[rows, 2:, 17] = True
            assert torch.equal(got[~hit], clean[~hit]), (new, i, hex(what))
            if what == 0x7FC0:
                assert torch.isnan(got[hit]).all()
            else:
                assert torch.isinf(got[hit]).all() and ((got[hit] > 0) == (what == 0x7F80)).all()


def test_a_request_of_too_many_rows_is_passed_over(wq):
    rng = np.random.default_rng(7)
    ctx, new = [40, 300], [8193, 3]
    c = Cache(rng, ctx, 1, 3, 64, 128, 128)
    n = sum(new)
    q, kv = bf16_bits(rng, n, 1, D), [bf16_bits(rng, n, 1, D) for _ in range(2)]
    parents = np.concatenate([np.arange(-1, 8192), [-1, 0, 0]])
    out = torch.full((n, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    wq.hlwq_kv_tree_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), i32(parents), i32([0, 8193, n]),
                              i32([t + m for t, m in zip(ctx, new)]), i32(c.table), *c.tensors(), out=out)
    got = out.cpu().double().numpy()
    assert np.all(got[:8193] == 7)
    r = slice(8193, n)
    check_tree(got[r], f64(q[r]), *sides(c, 1, 300, [x[r] for x in kv]), 300, parents[r], range(3))


def test_lengths_and_ranges_that_do_not_fit(wq):
    rng = np.random.default_rng(8)
    c = Cache(rng, [0], 2, 3, 64, 128, 128)
    q, kv = bf16_bits(rng, 5, 4, D), [bf16_bits(rng, 5, 2, D) for _ in range(2)]
    t, parents = (dev16(q), dev16(kv[0]), dev16(kv[1])), i32([-1, 0, 0, 1, 2])
    a = wq.hlwq_kv_tree_attention(*t, parents, i32([0, 5]), i32([5]), i32(c.table), *c.tensors())
    b = wq.hlwq_kv_tree_attention(*t, parents, i32([0, 5]), i32([-2 ** 31]), i32(c.table), *c.tensors())
    e = wq.hlwq_kv_tree_attention(*t, parents, i32([-7, 2000]), i32([5]), i32(c.table), *c.tensors())
    f = torch.full_like(a, 3.0)
    wq.hlwq_kv_tree_attention(*t, parents, i32([9, 2]), i32([5]), i32(c.table), *c.tensors(), out=f)
    assert torch.equal(a, b) and torch.equal(a, e) and bool((f == 3).all())


def test_given_workspace_is_enough_and_streams(wq):
    rng = np.random.default_rng(9)
    ctx, new = [300, 2000, 5], [9, 1, 20]
    c = Cache(rng, ctx, 2, 3, 64, 128, 128)
    n = sum(new)
    q, kv = bf16_bits(rng, n, 6, D), [bf16_bits(rng, n, 2, D) for _ in range(2)]
    t = [dev16(q), dev16(kv[0]), dev16(kv[1]), i32(trees(rng, new, 3)), i32([0, 9, 10, 30]), i32([309, 2001, 25]), i32(c.table),
         *c.tensors()]
    want = wq.hlwq_kv_tree_attention(*t)
    size = wq.hlwq_kv_tree_attention_workspace(3, n, 6, 2)
    ws = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [wq.hlwq_kv_tree_attention(*t, workspace=ws[:size] if i == 0 else None, stream=s) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got) and bool((ws[size:] == 255).all())
    with pytest.raises(wq.HLWQError):
        wq.hlwq_kv_tree_attention(*t, workspace=ws[:size - 16])
    with pytest.raises(ValueError):
        wq.hlwq_kv_tree_attention(*t[:3], t[3][:-1], *t[4:])
    with pytest.raises(TypeError):
        wq.hlwq_kv_tree_attention(*t[:3], t[3].long(), *t[4:])


def test_capture_and_replay(wq):
    rng = np.random.default_rng(10)
    ctx, new = [300, 70], [6, 4]
    c = Cache(rng, ctx, 2, 3, 64, 128, 128)
    q, kv = bf16_bits(rng, 10, 6, D), [bf16_bits(rng, 10, 2, D) for _ in range(2)]
    parents = i32(trees(rng, new, 3))
    t = [dev16(q), dev16(kv[0]), dev16(kv[1]), parents, i32([0, 6, 10]), i32([306, 74]), i32(c.table), *c.tensors()]
    ws = torch.empty(wq.hlwq_kv_tree_attention_workspace(2, 10, 6, 2), dtype=torch.uint8, device="cuda")
    wq.hlwq_kv_tree_attention(*t, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = wq.hlwq_kv_tree_attention(*t, workspace=ws)
    for _ in range(4):
        parents.copy_(i32(trees(rng, new, 3)))
        t[0].copy_(dev16(bf16_bits(rng, 10, 6, D)))
        want = wq.hlwq_kv_tree_attention(*t)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# Tiles of 64 rows: tables of 4000 tokens and more, 192 rows of a KV head and 48 a request.
def wide_case(wq, seed, ctx, new, q_heads, kv_heads, bits=3, page=64, **kw):
    rows = (sum(new) + kw.get("pad", 0)) * q_heads // kv_heads
    assert rows >= max(192, 48 * len(new))
    tree_case(wq, seed, ctx, new, q_heads, kv_heads, bits, page, width=max(4096 // page, (max(ctx) + page - 1) // page), **kw)


@pytest.mark.parametrize("ctx,new", [
    ([0], [192]), ([1], [33]), ([128], [35]), ([129], [40]), ([500], [64]), ([2049], [44]), ([5000], [64]), ([9000], [33]),
    ([0, 1, 15, 128, 129, 144, 145, 192, 193, 1000, 3000], [1, 2, 3, 4, 5, 60, 7, 8, 16, 17, 18]), ([1000, 30], [40, 0]),
    ([4000, 0, 999], [33, 1, 0]), ([96, 97, 127], [32, 31, 33]), ([4096, 4097, 6000, 65], [10, 11, 43, 1]),
])
@pytest.mark.parametrize("q_heads,kv_heads,bits,page", [(24, 4, 3, 64), (12, 2, 2, 16)])
def test_wide_lengths(wq, ctx, new, q_heads, kv_heads, bits, page):
    wide_case(wq, sum(ctx) + len(new), ctx, new, q_heads, kv_heads, bits, page)


@pytest.mark.parametrize("q_heads,kv_heads,new", [(1, 1, [200, 30]), (8, 8, [100, 92]), (8, 1, [9, 21]), (20, 4, [9, 31]), (17, 1, [9, 5])])
@pytest.mark.parametrize("bits", [3, 2])
def test_wide_heads(wq, q_heads, kv_heads, new, bits):
    wide_case(wq, q_heads, [333, 40], new, q_heads, kv_heads, bits, 32, wide=5)


@pytest.mark.parametrize("residual,ring", [(0, 0), (1, 1), (37, 37), (64, 100), (128, 1000)])
@pytest.mark.parametrize("bits,page,new", [(3, 16, [1, 50, 13]), (2, 256, [50, 10, 6])])
def test_wide_windows(wq, residual, ring, bits, page, new):
    wide_case(wq, residual + page, [residual + 50, 700, 20], new, 6, 2, bits, page, residual=residual, ring=ring)


@pytest.mark.parametrize("extra,pad", [(0, 5), (8, 0), (40, 30)])
def test_wide_strides_and_padding(wq, extra, pad):
    wide_case(wq, extra, [300, 3], [42, 27], 6, 2, extra=extra, pad=pad)


@pytest.mark.parametrize("scale,sigma", [(0.0, 1.0), (-1 / 16, 1.0), (1.0, 1.0), (1 / 16, 8.0)])
def test_wide_scales(wq, scale, sigma):
    wide_case(wq, 3, [300], [70], 6, 2, scale=scale, sigma=sigma)


@pytest.mark.parametrize("new,wide", [([1100, 257], 1), ([300], 1000)])
def test_wide_large_trees(wq, new, wide):
    wide_case(wq, wide, [200] * len(new), new, 2, 1, wide=wide)


@pytest.mark.parametrize("ctx", [20800, 45000])
@pytest.mark.parametrize("bits,page", [(3, 16), (2, 64)])
def test_wide_stretches_of_many_pages(wq, ctx, bits, page):
    """Page ids are read 32 blocks of 64 tokens at a time: 24 tiles over 232 workgroups, 34 and 73 blocks each."""
    wide_case(wq, ctx, [ctx], [64], 24, 1, bits, page)


def test_wide_many_requests(wq):
    # more of them than a wave looks through at once, empty ones among them
    rng = np.random.default_rng(16)
    ctx = [int(x) for x in rng.integers(0, 400, 75)]
    new = [0 if b in (0, 30, 64, 74) else int(x) for b, x in enumerate(rng.integers(6, 14, 75))]
    wide_case(wq, 16, ctx, new, 24, 4, 3, 32)


def test_wide_rows_left_alone_and_replayed(wq):
    """Rows of a request of too many nodes, outputs on two streams at once, and a captured call."""
    rng = np.random.default_rng(12)
    ctx, new = [40, 300, 4100], [8193, 3, 50]
    c = Cache(rng, ctx, 1, 3, 64, 128, 128)
    n = sum(new)
    cu = np.concatenate([[0], np.cumsum(new)])
    q, kv = bf16_bits(rng, n, 1, D), [bf16_bits(rng, n, 1, D) for _ in range(2)]
    parents = np.concatenate([np.arange(-1, 8192), trees(rng, new[1:], 3)])
    t = [dev16(q), dev16(kv[0]), dev16(kv[1]), i32(parents), i32(cu), i32([x + m for x, m in zip(ctx, new)]), i32(c.table), *c.tensors()]
    size = wq.hlwq_kv_tree_attention_workspace(3, n, 1, 1)
    ws = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.full((n, 1, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, s in enumerate(streams):
        wq.hlwq_kv_tree_attention(*t, out=outs[i], workspace=ws[:size] if i == 0 else None, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(*outs) and bool((ws[size:] == 255).all())
    got = outs[0].cpu().double().numpy()
    assert np.all(got[:8193] == 7)
    for b in (1, 2):
        r = slice(cu[b], cu[b + 1])
        check_tree(got[r], f64(q[r]), *sides(c, b, ctx[b], [x[r] for x in kv]), ctx[b], parents[r], range(0, new[b], 5))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = wq.hlwq_kv_tree_attention(*t, out=torch.full_like(outs[0], 7.0), workspace=ws)
    for _ in range(3):
        t[0].copy_(dev16(bf16_bits(rng, n, 1, D)))
        want = wq.hlwq_kv_tree_attention(*t, out=outs[1])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_wide_nan_and_infinities_stay_with_the_rows_that_see_them(wq):
    rng = np.random.default_rng(13)
    new, ctx = [70, 30], [300, 20]
    n = sum(new)
    c = Cache(rng, ctx, 2, 3, 64, 128, 128, width=64)
    q, kv = bf16_bits(rng, n, 4, D), [bf16_bits(rng, n, 2, D) for _ in range(2)]
    parents = trees(rng, new, 4)
    rest = (i32(parents), i32([0, new[0], n]), i32([t + m for t, m in zip(ctx, new)]), i32(c.table), *c.tensors())
    clean = wq.hlwq_kv_tree_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), *rest)
    ways = [way(parents[:new[0]], i) for i in range(new[0])]
    bad = max(range(1, new[0]), key=lambda x: sum(x in w for w in ways) % (new[0] - 1))
    rows = [i for i in range(new[0]) if bad in ways[i]]
    assert 1 < len(rows) < new[0] - 1
    for i, what in ((0, 0x7FC0), (1, 0x7FC0), (1, 0x7F80)):
        dirty = [x.copy() for x in kv]
        dirty[i][bad, 1, 17] = what
        got = wq.hlwq_kv_tree_attention(dev16(q), dev16(dirty[0]), dev16(dirty[1]), *rest)
        hit = torch.zeros(n, 4, D, dtype=torch.bool, device="cuda")
        hit[rows, 2:, slice(None) if i == 0 else 17] = True
        assert torch.equal(got[~hit], clean[~hit]), (i, hex(what))
        assert not torch.isfinite(got[hit]).any()


@pytest.mark.parametrize("new,width", [([12, 3], None), ([70, 30], 64)])
def test_a_bad_query_stays_in_its_row(wq, new, width):
    rng = np.random.default_rng(14)
    ctx, n = [300, 20], sum(new)
    c = Cache(rng, ctx, 2, 3, 64, 128, 128, width=width)
    q, kv = bf16_bits(rng, n, 4, D), [bf16_bits(rng, n, 2, D) for _ in range(2)]
    rest = (i32(trees(rng, new, 4)), i32([0, new[0], n]), i32([t + m for t, m in zip(ctx, new)]), i32(c.table), *c.tensors())
    clean = wq.hlwq_kv_tree_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), *rest)
    dirty = q.copy()
    dirty[3, 1, 200], dirty[n - 2, 2, 0] = 0x7FC0, 0x7F80
    got = wq.hlwq_kv_tree_attention(dev16(dirty), dev16(kv[0]), dev16(kv[1]), *rest)
    hit = torch.zeros(n, 4, dtype=torch.bool, device="cuda")
    hit[3, 1] = hit[n - 2, 2] = True
    assert torch.isnan(got[3, 1]).all() and not torch.isfinite(got[n - 2, 2]).any()
    assert torch.equal(got[~hit], clean[~hit])


def test_two_graphs_share_a_workspace(wq):
    """Captured calls with tiles of 64 rows and of 16 on one workspace, replayed in turn."""
    rng = np.random.default_rng(15)
    cases = []
    for ctx, new, width in (([4200, 70], [60, 40], None), ([300, 70], [6, 4], 8)):
        c, n = Cache(rng, ctx, 2, 3, 64, 128, 128, width=width), sum(new)
        q, kv = bf16_bits(rng, n, 6, D), [bf16_bits(rng, n, 2, D) for _ in range(2)]
        cases.append([dev16(q), dev16(kv[0]), dev16(kv[1]), i32(trees(rng, new, 3)), i32([0, new[0], n]),
                      i32([t + m for t, m in zip(ctx, new)]), i32(c.table), *c.tensors()])
    ws = torch.empty(max(wq.hlwq_kv_tree_attention_workspace(2, t[0].shape[0], 6, 2) for t in cases), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for t in cases:
        wq.hlwq_kv_tree_attention(*t, workspace=ws)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(wq.hlwq_kv_tree_attention(*t, workspace=ws))
    for _ in range(3):
        for t in cases:
            t[0].copy_(dev16(bf16_bits(rng, t[0].shape[0], 6, D)))
        wants = [wq.hlwq_kv_tree_attention(*t) for t in cases]
        for i in (1, 0, 0, 1):
            outs[i].zero_()
            graphs[i].replay()
            assert torch.equal(outs[i], wants[i])
            ws.fill_(255)


def test_steps_of_drafted_tokens(wq):
    """Trees through attention, an experts' layer and the verification; what is kept goes into the cache by plan and
    append, step after step, and every step's outputs are those of the definition on a cache built token by token."""
    rng = np.random.default_rng(11)
    heads, hq, page, residual, ring, bits = 2, 6, 16, 20, 40, 3
    ctx = [0, 55, 18]
    n, vocab, hidden, experts = 3, 96, hq * D, 8
    c = Cache(rng, ctx, heads, bits, page, residual, ring, spare=60, width=12)
    table, stack, n_free, tokens = i32(c.table), i32(c.stack), i32([c.n_free]), i32(ctx)
    cache = c.tensors()
    bank = [torch.from_numpy((rng.standard_normal(s) * 0.02).astype(np.float32)).to(torch.bfloat16).cuda()
            for s in ((experts, 2 * 64, hidden), (experts, hidden, 64))]
    up, down = wq.hlwq_quantize(bank[0]), wq.hlwq_quantize(bank[1])
    router = torch.from_numpy(rng.standard_normal((experts, hidden)).astype(np.float32)).to(torch.bfloat16).cuda()
    head = torch.from_numpy((rng.standard_normal((hidden, vocab)) * 0.2).astype(np.float32)).cuda()
    kept_total = 0
    for step in range(6):
        new = [int(x) for x in rng.integers(1, 12, n)]
        rows = sum(new) + 2
        cu = np.concatenate([[0], np.cumsum(new)])
        parents = np.concatenate([trees(rng, new, 3), [-1, -1]]).astype(np.int32)
        q, kv = bf16_bits(rng, rows, hq, D), [bf16_bits(rng, rows, heads, D) for _ in range(2)]
        dk, dv = dev16(kv[0]), dev16(kv[1])
        draft_ids = rng.integers(0, vocab, rows).astype(np.int32)
        held = tokens.cpu().numpy()
        out = wq.hlwq_kv_tree_attention(dev16(q), dk, dv, i32(parents), i32(cu), tokens + i32(new), table, *cache,
                                        n_residual=residual, bits=bits)
        y = wq.hlwq_moe_layer(out.view(rows, hidden).nan_to_num(), router, *up, *down, top_k=2).out
        p = torch.softmax((out.view(rows, hidden).nan_to_num() + y).float() @ head, -1)
        u, un = rng.random(rows).astype(np.float32), rng.random(n).astype(np.float32)
        qd = torch.full((rows, vocab), 1 / vocab, device="cuda")
        v = wq.hlwq_verify_drafts(i32(draft_ids), i32(parents), i32(cu), p, torch.from_numpy(u).cuda(), torch.from_numpy(un).cuda(),
                                  draft=qd)
        # the definition on the host's copy of the cache
        for i in range(2):
            c.packed[i], c.norms[i] = cache[2 * i].cpu().numpy(), cache[2 * i + 1].cpu().view(torch.int16).numpy().view(np.uint16)
            c.window[i] = cache[4 + i].cpu().view(torch.int16).numpy().view(np.uint16)
        c.table = table.cpu().numpy()
        got = out.cpu().double().numpy()
        for b in range(n):
            r = slice(cu[b], cu[b + 1])
            check_tree(got[r], f64(q[r]), *sides(c, b, int(held[b]), [x[r] for x in kv]), int(held[b]), parents[r], range(new[b]))
        want = vr.verify(draft_ids, parents, cu, p.double().cpu().numpy(), qd.double().cpu().numpy(), u, un)
        for a, b in zip(v, want):
            assert np.array_equal(a.cpu().numpy(), b)
        # what was kept, side by side, into the cache
        plan = wq.hlwq_kv_page_plan(tokens, v.n_kept, stack, n_free, table, rows, page_size=page, n_residual=residual)
        request = plan.row_request.clamp(min=0).long()
        place = (i32(cu)[request] + torch.arange(rows, device="cuda") - plan.cu_new[request]).clamp(0, rows - 1)
        source = torch.where(plan.row_request >= 0, v.kept[place], 0).long().clamp(min=0)
        wq.hlwq_kv_paged_append(dk[source], dv[source], plan.cu_new, plan.lens, plan.row_request, plan.slots, *cache,
                                n_residual=residual, bits=bits)
        assert plan.status.item() == 0
        tokens, n_free = plan.lens, plan.n_free
        assert np.array_equal(tokens.cpu().numpy(), held + want[0])
        kept_total += int(want[0].sum())
    assert kept_total > 18
