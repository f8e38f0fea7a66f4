"""GPU tests of the serving operators at the ends of their ranges: long chunks shared by many workgroups, batches that
mix chunks and single tokens, wide tiles of prompts, norms far apart, pools and rows past 4 GiB, shared pages, tables
of the largest width, and calls captured, replayed and put on other streams."""
import numpy as np
import pytest

import paged_ref as pr
from test_gpu_paged import Cache, D, attention_case, bf16_bits, dev16, f64, i32, prompt_case, wq  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# work shared by many workgroups
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("ctx,new,q_heads,kv_heads,bits,page,residual,ring", [
    ([3000], [300], 24, 4, 3, 64, 128, 128),
    ([4099], [130], 16, 2, 2, 16, 128, 300),
    ([2000, 700, 0], [101, 257, 64], 6, 2, 3, 256, 0, 0),
    ([900], [33], 1, 1, 3, 32, 200, 201),
    ([1000, 1000], [65, 64], 8, 8, 2, 128, 37, 37),
    ([333], [256], 1, 1, 3, 64, 128, 128),
    ([333], [257], 1, 1, 2, 64, 128, 128),
    ([0], [300], 6, 1, 3, 64, 128, 128),
])
def test_long_chunks(wq, ctx, new, q_heads, kv_heads, bits, page, residual, ring):
    attention_case(wq, sum(new), ctx, new, q_heads, kv_heads, bits, page, residual, ring, extra=8, pad=3)


@pytest.mark.parametrize("bits", [3, 2])
def test_chunks_and_single_tokens_in_one_batch(wq, bits):
    rng = np.random.default_rng(bits)
    ctx = [int(t) for t in rng.integers(0, 900, 70)]
    new = [int(rng.integers(17, 150)) if b % 9 == 0 else int(rng.integers(0, 3)) for b in range(70)]
    attention_case(wq, bits, ctx, new, 4, 2, bits, 32, 128, 128, pad=7)


def test_many_rows_of_few_tokens(wq):
    # sixteen and 32 rows to a tile, full and one past it
    for q_heads, n in ((16, 1), (17, 1), (32, 1), (16, 2), (8, 4), (11, 3)):
        attention_case(wq, q_heads, [1300, 5, 260], [n, n, n], q_heads, 1, 3, 64, 128, 128)


@pytest.mark.parametrize("count,q_heads,kv_heads", [(64, 16, 8), (65, 16, 8), (130, 16, 8), (64, 32, 16), (65, 16, 16)])
def test_wide_prompt_tiles(wq, count, q_heads, kv_heads):
    # enough tiles for those of 256 rows, the tiles of up to 64 sequences taken longest first
    rng = np.random.default_rng(count)
    lens = [int(n) for n in rng.integers(0, 100, count)]
    lens[3], lens[5], lens[count - 1] = 330, 257, 128
    prompt_case(wq, count, lens, q_heads, kv_heads, extra=8, pad=5)


@pytest.mark.parametrize("lens,q_heads,kv_heads", [([700], 6, 1), ([384], 4, 4), ([513, 300, 400], 5, 1), ([1100, 1], 2, 1)])
def test_prompt_tiles_with_keys_halved(wq, lens, q_heads, kv_heads):
    # few tiles of long sequences
    prompt_case(wq, sum(lens), lens, q_heads, kv_heads, extra=8, pad=2)


def test_halved_prompt_tiles_nan_and_infinities(wq):
    rng = np.random.default_rng(12)
    n = 450
    q, kv = bf16_bits(rng, n, 6, D), [bf16_bits(rng, n, 2, D) for _ in range(2)]
    cu = i32([0, n])
    clean = wq.hlwq_prompt_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), cu)
    for row in (0, 31, 32, 63, 64, 200, 449):
        for i, what in ((0, 0x7FC0), (1, 0x7FC0), (1, 0x7F80)):
            dirty = [x.copy() for x in kv]
            dirty[i][row, 1, 250] = what
            got = wq.hlwq_prompt_attention(dev16(q), dev16(dirty[0]), dev16(dirty[1]), cu)
            hit = torch.zeros(n, 6, D, dtype=torch.bool, device="cuda")
            hit[row:, 3:, slice(None) if i == 0 else 250] = True
            assert torch.equal(got[~hit], clean[~hit]), (row, i, hex(what))
            assert (torch.isnan(got[hit]) if what == 0x7FC0 else torch.isposinf(got[hit])).all()


@pytest.mark.parametrize("q_heads,kv_heads", [(16, 8), (32, 16)])
def test_wide_prompt_tiles_nan_and_infinities(wq, q_heads, kv_heads):
    rng = np.random.default_rng(11)
    lens = [200] + [60] * 63
    n = sum(lens)
    q, kv = bf16_bits(rng, n, q_heads, D), [bf16_bits(rng, n, kv_heads, D) for _ in range(2)]
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    clean = wq.hlwq_prompt_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), cu)
    for row, end in ((0, 200), (64, 200), (127, 200), (199, 200), (230, 260)):
        for i, what in ((0, 0x7FC0), (1, 0x7FC0), (1, 0xFF80)):
            dirty = [x.copy() for x in kv]
            dirty[i][row, 3, 40] = what
            got = wq.hlwq_prompt_attention(dev16(q), dev16(dirty[0]), dev16(dirty[1]), cu)
            hit = torch.zeros(n, q_heads, D, dtype=torch.bool, device="cuda")
            hit[row:end, 6:8, slice(None) if i == 0 else 40] = True
            assert torch.equal(got[~hit], clean[~hit]), (row, i, hex(what))
            assert (torch.isnan(got[hit]) if what == 0x7FC0 else torch.isneginf(got[hit])).all()


def test_chunks_nan_and_infinities(wq):
    rng = np.random.default_rng(5)
    ctx, new = [300, 20], [190, 100]
    n = sum(new)
    c = Cache(rng, ctx, 2, 3, 64, 128, 128)
    q, kv = bf16_bits(rng, n, 4, D), [bf16_bits(rng, n, 2, D) for _ in range(2)]
    cu, lens = i32([0, 190, 290]), i32([490, 120])
    clean = wq.hlwq_kv_paged_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), cu, lens, i32(c.table), *c.tensors())
    for row, end in ((0, 190), (63, 190), (64, 190), (189, 190), (200, 290)):
        for i, what in ((0, 0x7FC0), (1, 0x7FC0), (1, 0x7F80)):
            dirty = [x.copy() for x in kv]
            dirty[i][row, 1, 77] = what
            got = wq.hlwq_kv_paged_attention(dev16(q), dev16(dirty[0]), dev16(dirty[1]), cu, lens, i32(c.table), *c.tensors())
            hit = torch.zeros(n, 4, D, dtype=torch.bool, device="cuda")
            hit[row:end, 2:, slice(None) if i == 0 else 77] = True
            assert torch.equal(got[~hit], clean[~hit]), (row, i, hex(what))
            assert (torch.isnan(got[hit]) if what == 0x7FC0 else torch.isposinf(got[hit])).all()


@pytest.mark.parametrize("new", [[3, 2], [60, 40]])
def test_nan_in_a_query_stays_in_its_row(wq, new):
    rng = np.random.default_rng(3)
    ctx, n = [500, 300], sum(new)
    c = Cache(rng, ctx, 1, 3, 64, 128, 128)
    q, kv = bf16_bits(rng, n, 4, D), [bf16_bits(rng, n, 1, D) for _ in range(2)]
    dirty = q.copy()
    dirty[1, 2, 9] = 0x7FC0
    cu, lens = [0, new[0], n], i32([t + m for t, m in zip(ctx, new)])
    got = wq.hlwq_kv_paged_attention(dev16(dirty), dev16(kv[0]), dev16(kv[1]), i32(cu), lens, i32(c.table), *c.tensors())
    assert torch.isnan(got[1, 2]).all()
    got = got.cpu().double().numpy()
    clean = f64(q)
    for b in range(2):
        r = slice(cu[b], cu[b + 1])
        k, v = c.tokens_of(b, ctx[b], [x[r] for x in kv])
        mine = got[r].copy()
        if b == 0:  # the row itself was looked at above
            mine[1, 2] = pr.attend(clean[1, 2:3], k[0], v[0], ctx[0] + 2, 1 / 16, np.zeros(k.shape[1]), np.zeros(k.shape[1]))[0]
        pr.check_attention(mine, clean[r], k, v, pr.encoded(ctx[b], 128), ctx[b], 1)


@pytest.mark.parametrize("new", [1, 40, 300])
def test_norms_far_apart(wq, new):
    """The token that a row attends to most has a value 2^19 times smaller than the largest."""
    rng = np.random.default_rng(new)
    c = Cache(rng, [700], 1, 3, 64, 0, 0)
    v_norms = c.norms[1].view(np.float16)
    for t in range(700):
        v_norms[c.table[0, t // 64], 0, t % 64] = 2.0 ** -6 if t == 333 else 2.0 ** 13
    c.to_device()
    kv = [np.zeros((new, 1, D), np.uint16) for _ in range(2)]
    k, v = c.tokens_of(0, 700, kv)
    like = torch.from_numpy(k[0, 333][None, None] * np.ones((new, 1, 1)) * 2.0).to(torch.bfloat16)
    q = like.view(torch.int16).numpy().view(np.uint16)
    out = wq.hlwq_kv_paged_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), i32([0, new]), i32([700 + new]), i32(c.table),
                                     *c.tensors(), n_residual=0)
    pr.check_attention(out.cpu().double().numpy(), f64(q), k, v, 700, 700, 1)


# ---------------------------------------------------------------------------
# offsets past 32 bits: the same contents in a small and in a large buffer
# ---------------------------------------------------------------------------

def test_pages_past_4_gib(wq):
    rng = np.random.default_rng(21)
    pages, heads, page = 180_000, 4, 64  # 4.4 GB of 3-bit codes
    c = Cache(rng, [1100, 300], heads, 3, page, 128, 128, spare=20)
    to = torch.from_numpy(rng.permutation(pages - 1000)[:c.pool] + 1000).cuda()
    to[:4] = torch.tensor([pages - 1, pages - 2, 0, 175_000], device="cuda")
    big = [torch.empty(pages, heads, page, 96, dtype=torch.uint8, device="cuda"),
           torch.empty(pages, heads, page, dtype=torch.float16, device="cuda")]
    big += [torch.empty_like(x) for x in big]
    assert big[0].numel() > 2 ** 32
    for x, y in zip(big, c.d):
        x[to] = y
    small, small_table = c.tensors(), i32(c.table)
    windows = [x.clone() for x in small[4:]]
    table = torch.where(small_table >= 0, to.int()[small_table.clamp(min=0).long()], small_table)
    for new in ([1, 1], [40, 30]):
        n = sum(new)
        q, k, v = (dev16(bf16_bits(rng, n, h, D)) for h in (12, heads, heads))
        cu, lens = i32([0, new[0], n]), i32([1100 + new[0], 300 + new[1]])
        want = wq.hlwq_kv_paged_attention(q, k, v, cu, lens, small_table, *small)
        got = wq.hlwq_kv_paged_attention(q, k, v, cu, lens, table, *big, *windows)
        assert torch.equal(want, got), new
    # the same rows appended to both: the pushed-out tokens go to the pages numbered 0 .. c.pool - 1 here
    n = 70
    k, v = (dev16(bf16_bits(rng, n, heads, D)) for _ in range(2))
    at = torch.arange(n, device="cuda")
    ids, offs = at % c.pool, (at * 7) % page
    req = i32([0] * 40 + [1] * 30)
    cu, lens = i32([0, 40, 70]), i32([1140, 330])
    wq.hlwq_kv_paged_append(k, v, cu, lens, req, (ids * page + offs).int(), *small)
    wq.hlwq_kv_paged_append(k, v, cu, lens, req, (to[ids] * page + offs).int(), *big, *windows)
    for x, y in zip([b[to] for b in big] + windows, small):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_windows_and_rows_past_4_gib(wq):
    rng = np.random.default_rng(22)
    c = Cache(rng, [700, 400], 2, 3, 64, 128, 128)
    ring = 2 ** 20 + 129  # 2 GiB a request, K and V each
    far = [torch.empty(2, 2, ring, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert far[0].numel() * 2 > 2 ** 31
    for i, x in enumerate(far):
        for b, t in enumerate((700, 400)):
            s = torch.arange(t - 128, t, device="cuda")
            x[b][:, s % ring] = c.d[4 + i][b][:, s % 128]
    for new in ([1, 1], [50, 33]):
        n = sum(new)
        bits = [bf16_bits(rng, n, h, D) for h in (6, 2, 2)]
        near = [dev16(x) for x in bits]
        stride = 2 ** 22
        wide = []
        for x in near:
            pool = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda")
            rows = pool.as_strided(x.shape, (stride, D, 1))
            rows.copy_(x)
            wide.append(rows)
        cu, lens = i32([0, new[0], n]), i32([700 + new[0], 400 + new[1]])
        want = wq.hlwq_kv_paged_attention(*near, cu, lens, i32(c.table), *c.tensors())
        got = wq.hlwq_kv_paged_attention(*wide, cu, lens, i32(c.table), *c.d[:4], *far)
        assert torch.equal(want, got), new
        assert torch.equal(wq.hlwq_prompt_attention(*near, cu), wq.hlwq_prompt_attention(*wide, cu)), new


@pytest.mark.parametrize("new,q_heads", [(300, 24), (1, 4)])
def test_the_widest_table(wq, new, q_heads):
    """2^20 entries of 256 tokens, nearly all of them beyond the request."""
    rng = np.random.default_rng(new)
    c = Cache(rng, [900], 4, 3, 256, 128, 128, width=2 ** 20 - 4)
    q, k, v = (bf16_bits(rng, new, h, D) for h in (q_heads, 4, 4))
    out = wq.hlwq_kv_paged_attention(dev16(q), dev16(k), dev16(v), i32([0, new]), i32([900 + new]), i32(c.table), *c.tensors())
    keys = c.tokens_of(0, 900, [k, v])
    pr.check_attention(out.cpu().double().numpy(), f64(q), *keys, pr.encoded(900, 128), 900, 4)


# ---------------------------------------------------------------------------
# use
# ---------------------------------------------------------------------------

def test_requests_may_share_pages(wq):
    rng = np.random.default_rng(31)
    c = Cache(rng, [640, 640], 2, 3, 64, 128, 128)
    for x in c.d[4:]:
        x[1] = x[0]
    table = i32(c.table)
    table[1] = table[0]
    for new in (1, 40):
        bits = [bf16_bits(rng, new, h, D) for h in (4, 2, 2)]
        q, k, v = (dev16(x).repeat(2, 1, 1) for x in bits)
        out = wq.hlwq_kv_paged_attention(q, k, v, i32([0, new, 2 * new]), i32([640 + new] * 2), table, *c.tensors())
        # Both requests against the definition, not element by element against each other: their work is cut at other
        # places, so a probability p is rounded (2^-8 p to bf16, 2^-11 p n to fp16) over another running maximum, and an
        # element, a sum of 680 such terms of either sign, may differ by the sum of those roundings, 2^-8 sum_j p_j |v_j|
        # for each call, however small the element itself is.  That is the bound that check_attention takes.
        keys = c.tokens_of(0, 640, bits[1:])
        for rows in (out[:new], out[new:]):
            pr.check_attention(rows.cpu().double().numpy(), f64(bits[0]), *keys, pr.encoded(640, 128), 640, 2)


def test_captured_chunks_and_prompts_replay(wq):
    rng = np.random.default_rng(33)
    c = Cache(rng, [700, 300], 2, 3, 64, 128, 128)
    q, k, v = (torch.zeros(90, h, D, dtype=torch.bfloat16, device="cuda") for h in (6, 2, 2))
    cu, lens, table = i32([0, 50, 90]), i32([750, 340]), i32(c.table)
    work = torch.empty(wq.hlwq_kv_paged_attention_workspace(2, 90, 6, 2), dtype=torch.uint8, device="cuda")

    def run():
        return (wq.hlwq_kv_paged_attention(q, k, v, cu, lens, table, *c.tensors(), workspace=work),
                wq.hlwq_prompt_attention(q, k, v, cu))

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for new in ([50, 40], [1, 1], [89, 0], [0, 0], [3, 87]):
        for x in (q, k, v):
            x.copy_(dev16(bf16_bits(rng, *x.shape)))
        cu.copy_(i32([0, new[0], sum(new)]))
        lens.copy_(i32([700 + new[0], 300 + new[1]]))
        want = [x.clone() for x in run()]
        work.fill_(0xFF)  # NaN, whatever the call before left
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(w[:sum(new)], h[:sum(new)]) for w, h in zip(want, held)), new
        torch.rand(1 << 20, device="cuda").sum().item()


def test_every_call_on_another_stream(wq):
    rng = np.random.default_rng(35)
    here, there = [Cache(np.random.default_rng(1), [500, 130, 0], 2, 3, 16, 128, 128, spare=30, width=60) for _ in range(2)]
    new = [40, 1, 20]
    q, k, v = (dev16(bf16_bits(rng, 61, h, D)) for h in (4, 2, 2))

    def step(c, stream):
        table, free = i32(c.table), i32(c.stack)
        args = (i32(c.ctx), i32(new), free, i32([c.n_free]), table)
        torch.cuda.synchronize()
        p = wq.hlwq_kv_page_plan(*args, 61, page_size=16, stream=stream)
        a = wq.hlwq_kv_paged_attention(q, k, v, p.cu_new, p.lens, table, *c.tensors(), stream=stream)
        b = wq.hlwq_prompt_attention(q, k, v, p.cu_new, stream=stream)
        wq.hlwq_kv_paged_append(k, v, p.cu_new, p.lens, p.row_request, p.slots, *c.tensors(), stream=stream)
        torch.cuda.synchronize()
        return [*p, a, b, table, free, *c.d]

    for x, y in zip(step(here, None), step(there, torch.cuda.Stream())):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("new", [[1, 1], [3, 0], [200, 150]])
def test_no_pages_at_all(wq, new):
    """A pool of no pages and tables of no entries: encoded tokens are left out, window and own tokens are not."""
    rng = np.random.default_rng(41)
    c = Cache(rng, [300, 50], 2, 3, 64, 128, 128)
    n = sum(new)
    q, kv = bf16_bits(rng, n, 4, D), [bf16_bits(rng, n, 2, D) for _ in range(2)]
    none = [torch.zeros(0, 2, 64, 96, dtype=torch.uint8, device="cuda"), torch.zeros(0, 2, 64, dtype=torch.float16, device="cuda")]
    table = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    cu, lens = [0, new[0], n], i32([300 + new[0], 50 + new[1]])
    out = wq.hlwq_kv_paged_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), i32(cu), lens, table, *none, *none, *c.d[4:])
    got = out.cpu().double().numpy()
    for b, held in enumerate((300, 50)):
        r, enc = slice(cu[b], cu[b + 1]), pr.encoded(held, 128)
        if new[b]:
            k, v = (x[:, enc:] for x in c.tokens_of(b, held, [x[r] for x in kv]))
            pr.check_attention(got[r], f64(q[r]), k, v, 0, held - enc, 2)


def test_nothing_to_do(wq):
    c = Cache(np.random.default_rng(42), [300, 50], 2, 3, 64, 128, 128)
    before = [x.clone() for x in c.d]
    no = [torch.zeros(0, h, D, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2)]
    cu, lens, table = i32([0, 0, 0]), i32([300, 50]), i32(c.table)
    assert wq.hlwq_kv_paged_attention(*no, cu, lens, table, *c.tensors()).shape == (0, 4, D)
    assert wq.hlwq_prompt_attention(*no, cu).shape == (0, 4, D)
    wq.hlwq_kv_paged_append(*no[1:], cu, lens, cu[:0], cu[:0], *c.tensors())
    # rows that nobody owns are left as they were
    rows = [torch.ones(3, h, D, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2)]
    out = torch.full((3, 4, D), 5.0, dtype=torch.bfloat16, device="cuda")
    wq.hlwq_kv_paged_attention(*rows, cu, lens, table, *c.tensors(), out=out)
    wq.hlwq_prompt_attention(*rows, cu, out=out)
    wq.hlwq_prompt_attention(*rows, i32([0]), out=out)
    wq.hlwq_kv_paged_append(*rows[1:], cu, lens, i32([-1] * 3), i32([-1] * 3), *c.tensors())
    torch.cuda.synchronize()
    assert bool((out == 5).all())
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(before, c.d))


def test_same_call_twice_gives_the_same_bits(wq):
    rng = np.random.default_rng(43)
    c = Cache(rng, [900, 2000, 64], 2, 2, 32, 128, 128)
    for new in ([1, 1, 1], [90, 1, 200]):
        n = sum(new)
        q, k, v = (dev16(bf16_bits(rng, n, h, D)) for h in (12, 2, 2))
        cu, lens = i32(np.concatenate([[0], np.cumsum(new)])), i32([900 + new[0], 2000 + new[1], 64 + new[2]])
        first = wq.hlwq_kv_paged_attention(q, k, v, cu, lens, i32(c.table), *c.tensors(), bits=2)
        prompt = wq.hlwq_prompt_attention(q, k, v, cu)
        for _ in range(5):
            assert torch.equal(first, wq.hlwq_kv_paged_attention(q, k, v, cu, lens, i32(c.table), *c.tensors(), bits=2))
            assert torch.equal(prompt, wq.hlwq_prompt_attention(q, k, v, cu))
