"""GPU tests of the serving operators against plain CPU forms (tests/paged_ref.py).

Plan and append have to be equal bit for bit, what they do not write included.
Attention is compared with its 64-bit definition under a bound that counts the
roundings of its operands (paged_ref.attend).
"""
import numpy as np
import pytest

import paged_ref as pr

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

D = 256


@pytest.fixture(scope="module")
def wq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import weight_quantization_amd as m
    m.load_library()
    return m


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def dev16(bits, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(dtype).cuda()


def host16(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def bf16_bits(rng, *shape, sigma=1.0):
    return host16((torch.from_numpy(rng.standard_normal(shape).astype(np.float32)) * sigma).to(torch.bfloat16))


def f64(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def strided(bits, extra):
    """Rows [rows, heads, 256] as a slice of wider ones."""
    t = dev16(bits)
    wide = torch.full((t.shape[0], t.shape[1] * D + extra), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + t.shape[1] * D] = t.flatten(1)
    return wide[:, 8:8 + t.shape[1] * D].view(t.shape)


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------

def run_plan(wq, tokens, n_new, reset, stack, n_free, table, rows, page, residual):
    d_stack, d_table = i32(stack), i32(table)
    p = wq.hlwq_kv_page_plan(i32(tokens), i32(n_new), d_stack, i32([n_free]), d_table, rows, page_size=page,
                             n_residual=residual,
                             reset=None if reset is None else torch.tensor(np.asarray(reset), dtype=torch.uint8).cuda())
    torch.cuda.synchronize()
    return p, d_stack.cpu().numpy(), d_table.cpu().numpy()


def check_plan(wq, tokens, n_new, reset, stack, n_free, table, rows, page, residual):
    """Plans on the device and in Python, compares everything, and leaves the step done in stack and table."""
    tokens, n_new = [int(t) for t in tokens], [int(n) for n in n_new]
    p, d_stack, d_table = run_plan(wq, tokens, n_new, reset, stack, n_free, table, rows, page, residual)
    gone = [0] * len(tokens) if reset is None else reset
    want = pr.plan(tokens, n_new, gone, stack, n_free, table, rows, page, residual)
    for name, got, ref in zip(p._fields, p, want):
        assert np.array_equal(got.cpu().numpy().ravel(), np.ravel(ref)), name
    assert np.array_equal(d_stack, stack) and np.array_equal(d_table, table)
    return want


@pytest.mark.parametrize("B,page,residual,most,width", [
    (1, 64, 128, 300, 20), (3, 16, 0, 40, 30), (64, 64, 128, 90, 12), (257, 32, 37, 50, 9), (1024, 16, 128, 33, 20),
    (1025, 128, 64, 40, 6), (5000, 256, 1, 9, 4),
])
def test_plan_steps(wq, B, page, residual, most, width):
    rng = np.random.default_rng(B + page)
    pool = min(B * width, 60 * B)
    stack = np.full(pool, -1, np.int32)
    n_free = pool
    stack[:] = rng.permutation(pool)
    table = np.full((B, width), -1, np.int32)
    tokens = np.zeros(B, int)
    for step in range(6):
        reset = (rng.random(B) < 0.2) & (step > 0)
        held = np.where(reset, 0, tokens)
        n_new = np.where(rng.random(B) < 0.3, 0, rng.integers(0, most + 1, B))
        n_new = np.maximum(np.minimum(n_new, residual + (width * page) - held), 0)
        rows = int(n_new.sum()) + (0, 5, 300)[step % 3]
        cu, lens, *_, n_free, status = check_plan(wq, tokens, n_new, reset if step % 2 else (reset if reset.any() else None),
                                                  stack, n_free, table, rows, page, residual)
        assert status == 0
        tokens = lens.astype(int)
    assert n_free >= 0


def test_plan_can_be_repeated(wq):
    rng = np.random.default_rng(5)
    tokens, n_new, stack = rng.integers(0, 900, 9), rng.integers(0, 200, 9), rng.permutation(300)
    table = np.full((9, 40), -1)
    for b in range(9):
        table[b, :-(-max(tokens[b] - 128, 0) // 16) or None] = 0
    d = [i32(tokens), i32(n_new), i32(stack), i32([300]), i32(table)]
    a = wq.hlwq_kv_page_plan(*d, int(n_new.sum()) + 3, page_size=16)
    first = [t.clone() for t in (*a, *d)]
    b = wq.hlwq_kv_page_plan(*d, int(n_new.sum()) + 3, page_size=16)
    for x, y in zip(first, (*b, *d)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("fault,status", [
    (dict(n_new=[200, 64, 64]), None), (dict(tokens=[-1, 5, 5]), -1), (dict(n_new=[1, -2, 1]), -1), (dict(rows=2), -1),
    (dict(n_free=-1), -1), (dict(n_free=9), -1), (dict(tokens=[16 * 6 + 3, 0, 0], residual=0), -1),
    (dict(tokens=[2 ** 31 - 1, 0, 0], residual=2 ** 31 - 1), -1),
    (dict(reset=[1, 0, 0], tokens=[40, 0, 0], residual=0, bad_id=8), -1),
    (dict(reset=[1, 0, 0], tokens=[40, 0, 0], residual=0, bad_id=-1), -1),
    (dict(reset=[1, 0, 0], tokens=[40, 0, 0], residual=0, n_free=6), -1),
])
def test_plan_that_fails_changes_nothing(wq, fault, status):
    stack, table = np.arange(8, dtype=np.int32)[::-1].copy(), np.zeros((3, 5), np.int32)
    table[:] = np.arange(5)
    if "bad_id" in fault:
        table[0, 1] = fault["bad_id"]
    s0, t0 = stack.copy(), table.copy()
    n_free = fault.get("n_free", 4)
    tokens, residual = fault.get("tokens", [3, 2, 1]), fault.get("residual", 8)
    *_, n_after, got = check_plan(wq, tokens, fault.get("n_new", [1, 1, 1]), fault.get("reset"), stack, n_free, table,
                                  fault.get("rows", 400), 16, residual)
    assert got != 0 and (status is None or got == status) and n_after == n_free
    assert np.array_equal(stack, s0) and np.array_equal(table, t0)


def test_plan_of_nothing(wq):
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    p = wq.hlwq_kv_page_plan(none, none, none, i32([0]), none.view(0, 5), 4)
    assert p.cu_new.tolist() == [0] and p.row_request.tolist() == [-1] * 4 and p.status.item() == 0
    p = wq.hlwq_kv_page_plan(i32([0, 0]), i32([0, 0]), i32([0]), i32([1]), i32([[0], [0]]), 0)
    assert p.cu_new.tolist() == [0, 0, 0] and p.status.item() == 0 and p.n_free.item() == 1


# ---------------------------------------------------------------------------
# a cache in use
# ---------------------------------------------------------------------------

class Cache:
    """A paged cache on the host and on the device, with requests of given lengths in it; slots of the pool that hold
    no token hold NaN norms, and so does what the windows hold of nobody."""

    def __init__(self, rng, ctx, heads, bits, page, residual, ring, spare=3, width=None):
        self.ctx, self.heads, self.bits, self.page, self.residual, self.ring = ctx, heads, bits, page, residual, ring
        n = len(ctx)
        used = [-(-pr.encoded(t, residual) // page) for t in ctx]
        self.pool = sum(used) + spare
        self.width = max([*used, 1]) + (4 if width is None else width)
        ids = rng.permutation(self.pool)
        self.table = np.full((n, self.width), -1, np.int32)
        self.stack = np.full(self.pool, -1, np.int32)
        k = 0
        for b in range(n):
            self.table[b, :used[b]] = ids[k:k + used[b]]
            k += used[b]
        self.n_free = self.pool - k
        self.stack[:self.n_free] = ids[k:]
        self.packed, self.norms, self.window = [], [], []
        for _ in range(2):
            self.packed.append(rng.integers(0, 256, (self.pool, heads, page, 32 * bits), dtype=np.uint8))
            norms = np.full((self.pool, heads, page), np.nan, np.float16)
            for b in range(n):
                for t in range(pr.encoded(ctx[b], residual)):
                    norms[self.table[b, t // page], :, t % page] = rng.uniform(8, 24, heads)
            self.norms.append(norms.view(np.uint16))
            w = np.full((n, heads, ring, D), 0x7FC0, np.uint16)
            for b in range(n):
                at = np.arange(pr.encoded(ctx[b], residual), ctx[b]) % max(ring, 1)
                w[b][:, at] = bf16_bits(rng, heads, len(at), D)
            self.window.append(w)
        self.to_device()

    def to_device(self):
        self.d = [x for i in range(2) for x in (torch.from_numpy(self.packed[i].copy()).cuda(),
                                                dev16(self.norms[i], torch.float16))]
        self.d += [dev16(w) for w in self.window]

    def tensors(self):
        return self.d if self.ring or self.residual else [*self.d[:4], None, None]

    def same(self):
        """Whether the device holds exactly what the host does."""
        got = [self.d[0].cpu().numpy(), host16(self.d[1]), self.d[2].cpu().numpy(), host16(self.d[3]), host16(self.d[4]),
               host16(self.d[5])]
        want = [self.packed[0], self.norms[0], self.packed[1], self.norms[1], self.window[0], self.window[1]]
        return [np.array_equal(g, w) for g, w in zip(got, want)]

    def tokens_of(self, b, held, new):
        """Keys and values of request b in 64 bits, [heads, tokens, 256] each; new: the step's bf16 bits, K and V."""
        out = []
        for i in range(2):
            enc = pr.encoded(held, self.residual)
            t = np.arange(enc)
            ids = self.table[b, t // self.page]
            old = pr.decoded(self.packed[i][ids, :, t % self.page], self.norms[i][ids, :, t % self.page].view(np.float16),
                             self.bits) if enc else np.zeros((0, self.heads, D))
            near = np.arange(enc, held)
            win = f64(self.window[i][b][:, near % max(self.ring, 1)]).transpose(1, 0, 2) if held > enc else old[:0]
            out.append(np.concatenate([old, win, f64(new[i])]).transpose(1, 0, 2))
        return out


APPENDS = [
    # ctx, new, residual, ring, page, heads, bits
    ([0], [1], 128, 128, 64, 4, 3),
    ([127, 128, 129, 5000], [1, 1, 1, 1], 128, 128, 64, 4, 3),
    ([500, 3, 0, 700], [1, 0, 5, 2], 128, 144, 16, 2, 2),
    ([0, 0], [1000, 77], 128, 128, 64, 2, 3),
    ([130, 1], [400, 300], 128, 128, 32, 1, 3),        # the step passes the whole ring
    ([130, 1, 64], [300, 200, 129], 128, 130, 32, 1, 2),  # a ring a little longer than the window
    ([90, 200], [64, 128], 128, 256, 16, 3, 3),
    ([40, 7], [5, 20], 0, 0, 16, 2, 3),                # no window
    ([40, 7], [5, 20], 0, 3, 16, 2, 2),                # a ring that nothing enters
    ([9, 30], [1, 40], 1, 1, 128, 5, 3),
    ([700], [90], 37, 50, 256, 1, 2),
    ([700, 20], [33, 34], 31, 37, 16, 7, 3),
]


@pytest.mark.parametrize("ctx,new,residual,ring,page,heads,bits", APPENDS)
@pytest.mark.parametrize("extra,pad", [(0, 0), (24, 3)])
def test_append(wq, ctx, new, residual, ring, page, heads, bits, extra, pad):
    rng = np.random.default_rng(sum(ctx) + sum(new) + ring)
    spare = sum(-(-(t + n) // page) for t, n in zip(ctx, new)) + 2
    c = Cache(rng, ctx, heads, bits, page, residual, ring, spare=spare, width=spare)
    rows = sum(new) + pad
    bits_new = [bf16_bits(rng, rows, heads, D) for _ in range(2)]
    bits_new[0][0, 0] = 0  # a zero vector
    cu, lens, req, _, slots, _, status = pr.plan(ctx, new, [0] * len(ctx), c.stack, c.n_free, c.table, rows, page, residual)
    assert status == 0
    t = [strided(x, extra) if extra else dev16(x) for x in bits_new]
    wq.hlwq_kv_paged_append(*t, i32(cu), i32(lens), i32(req), i32(slots), *c.tensors(), n_residual=residual, bits=bits)
    torch.cuda.synchronize()
    for i in range(2):
        pr.append(bits_new[i], cu, lens, req, slots, c.packed[i], c.norms[i], c.window[i], residual, bits)
    assert c.same() == [True] * 6


def test_append_passes_over_what_is_out_of_range(wq):
    rng = np.random.default_rng(3)
    c = Cache(rng, [300, 300, 300], 2, 3, 16, 128, 128)
    new = [bf16_bits(rng, 6, 2, D) for _ in range(2)]
    cu, lens = np.array([0, 2, 4, 6]), np.array([302, 302, 302])
    req, slots = np.array([0, 7, -3, 1, 2, 2]), np.array([0, 1, 2, 3, c.pool * 16, -9])
    wq.hlwq_kv_paged_append(dev16(new[0]), dev16(new[1]), i32(cu), i32(lens), i32(req), i32(slots), *c.tensors())
    torch.cuda.synchronize()
    ok = np.array([0, -1, -1, 1, 2, 2])
    slots = np.array([0, -1, -1, 3, -1, -1])
    for i in range(2):
        pr.append(new[i], cu, lens, ok, slots, c.packed[i], c.norms[i], c.window[i], 128, 3)
    assert c.same() == [True] * 6
    # rows of a request whose range is elsewhere, and ranges that leave the rows
    before = [x.clone() for x in c.d]
    wq.hlwq_kv_paged_append(dev16(new[0]), dev16(new[1]), i32([6, 6, 6, 6]), i32(lens), i32(req), i32(slots), *c.tensors())
    wq.hlwq_kv_paged_append(dev16(new[0]), dev16(new[1]), i32([-4, -4, -4, -9]), i32(lens), i32(req), i32(slots), *c.tensors())
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(before, c.d))


# ---------------------------------------------------------------------------
# paged attention
# ---------------------------------------------------------------------------

def attention_case(wq, seed, ctx, new, q_heads, kv_heads, bits, page, residual, ring, extra=0, pad=0, scale=1 / 16,
                   sigma=1.0):
    rng = np.random.default_rng(seed)
    c = Cache(rng, ctx, kv_heads, bits, page, residual, ring)
    rows = sum(new) + pad
    q = bf16_bits(rng, rows, q_heads, D, sigma=sigma)
    kv = [bf16_bits(rng, rows, kv_heads, D) for _ in range(2)]
    cu = np.concatenate([[0], np.cumsum(new)])
    out = torch.full((rows, q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    make = (lambda x: strided(x, extra)) if extra else dev16
    wq.hlwq_kv_paged_attention(make(q), make(kv[0]), make(kv[1]), i32(cu), i32([t + n for t, n in zip(ctx, new)]),
                               i32(c.table), *c.tensors(), n_residual=residual, bits=bits, scale=scale, out=out)
    torch.cuda.synchronize()
    got = out.cpu().double().numpy()
    worst = 0
    for b, (t, n) in enumerate(zip(ctx, new)):
        if not n:
            continue
        r = slice(cu[b], cu[b + 1])
        k, v = c.tokens_of(b, t, [x[r] for x in kv])
        worst = max(worst, pr.check_attention(got[r], f64(q[r]), k, v, pr.encoded(t, residual), t, kv_heads, scale))
    assert np.all(got[cu[-1]:] == 7.0)
    print(f"largest error {worst:.3f} of its bound", flush=True)


@pytest.mark.parametrize("ctx,new", [
    ([0], [1]), ([1], [1]), ([128], [1]), ([129], [1]), ([500], [1]), ([2049], [1]), ([5000], [1]),
    ([0, 1, 15, 16, 17, 127, 128, 129, 143, 144, 145, 191, 192, 193], [1] * 14),
    ([300, 0, 999], [0, 3, 2]), ([1000, 30], [5, 6]), ([400], [31]), ([260, 800], [65, 1]),
])
@pytest.mark.parametrize("q_heads,kv_heads,bits,page", [(24, 4, 3, 64), (6, 2, 2, 16)])
def test_attention_lengths(wq, ctx, new, q_heads, kv_heads, bits, page):
    attention_case(wq, sum(ctx) + len(new), ctx, new, q_heads, kv_heads, bits, page, 128, 128)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (8, 8), (16, 2), (8, 1), (12, 4), (10, 2), (17, 1), (33, 1), (64, 2)])
@pytest.mark.parametrize("bits", [3, 2])
def test_attention_heads(wq, q_heads, kv_heads, bits):
    attention_case(wq, q_heads, [700, 33], [2, 1], q_heads, kv_heads, bits, 64, 128, 128)


@pytest.mark.parametrize("residual,ring", [(0, 0), (0, 9), (1, 1), (37, 37), (64, 100), (128, 128), (128, 1000), (600, 600)])
@pytest.mark.parametrize("bits,page,new", [(3, 16, [1, 1, 1]), (2, 256, [3, 1, 2]), (3, 128, [20, 1, 33])])
def test_attention_windows(wq, residual, ring, bits, page, new):
    attention_case(wq, residual + ring, [555, 38, 100], new, 12, 2, bits, page, residual, ring)


@pytest.mark.parametrize("extra,pad", [(24, 0), (8, 5)])
def test_attention_strides_and_padding(wq, extra, pad):
    attention_case(wq, 1, [900, 70], [3, 1], 24, 4, 3, 64, 128, 128, extra=extra, pad=pad)
    attention_case(wq, 2, [900, 70], [50, 9], 6, 1, 2, 64, 128, 128, extra=extra, pad=pad)


@pytest.mark.parametrize("scale,sigma", [(1 / 16, 8.0), (1.0, 0.01), (-0.05, 1.0), (0.0, 1.0), (1 / 16, 300.0)])
def test_attention_scales(wq, scale, sigma):
    attention_case(wq, 3, [900, 70], [2, 1], 6, 1, 3, 64, 128, 128, scale=scale, sigma=sigma)


def test_attention_many_requests(wq):
    rng = np.random.default_rng(9)
    ctx = [int(t) for t in rng.integers(0, 400, 150)]
    attention_case(wq, 9, ctx, [int(n) for n in rng.integers(0, 4, 150)], 4, 1, 3, 32, 128, 128)
    attention_case(wq, 10, [0] * 700 + [129], [1] * 700 + [0], 2, 1, 2, 32, 128, 128)


def test_attention_skips_pages_that_are_not_there(wq):
    rng = np.random.default_rng(4)
    c = Cache(rng, [400, 400], 2, 3, 16, 128, 128)
    q, kv = bf16_bits(rng, 2, 4, D), [bf16_bits(rng, 2, 2, D) for _ in range(2)]
    table = c.table.copy()
    table[0, 2], table[0, 5], table[1, 0] = -1, c.pool, 2 ** 31 - 1
    args = (dev16(q), dev16(kv[0]), dev16(kv[1]), i32([0, 1, 2]), i32([401, 401]))
    out = wq.hlwq_kv_paged_attention(*args, i32(table), *c.tensors())
    short = wq.hlwq_kv_paged_attention(*args, i32(c.table[:, :3]), *c.tensors())
    torch.cuda.synchronize()
    for got, gone in ((out, [[2, 5], [0]]), (short, [range(3, 17)] * 2)):
        got = got.cpu().double().numpy()
        for b in range(2):
            k, v = c.tokens_of(b, 400, [x[b:b + 1] for x in kv])
            keep = ~np.isin(np.arange(401) // 16, [p for p in gone[b]]) | (np.arange(401) >= 272)
            pr.check_attention(got[b:b + 1], f64(q[b:b + 1]), k[:, keep], v[:, keep], int(keep[:272].sum()),
                               int(keep.sum()) - 1, 2)


def test_attention_nan_and_infinities_stay_with_the_rows_that_see_them(wq):
    rng = np.random.default_rng(6)
    for new in ([6, 3], [40, 21]):
        ctx, n = [300, 20], sum(new)
        c = Cache(rng, ctx, 2, 3, 64, 128, 128)
        q, kv = bf16_bits(rng, n, 4, D), [bf16_bits(rng, n, 2, D) for _ in range(2)]
        cu = [0, new[0], n]
        lens = i32([t + m for t, m in zip(ctx, new)])
        clean = wq.hlwq_kv_paged_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), i32(cu), lens, i32(c.table), *c.tensors())
        last = new[0] - 2  # the row of request 0 from which on NaN is seen
        for i, what in ((0, 0x7FC0), (1, 0x7FC0), (1, 0x7F80), (1, 0xFF80)):
            dirty = [x.copy() for x in kv]
            dirty[i][last, 1, 17] = what
            got = wq.hlwq_kv_paged_attention(dev16(q), dev16(dirty[0]), dev16(dirty[1]), i32(cu), lens, i32(c.table),
                                             *c.tensors())
            hit = torch.zeros(n, 4, D, dtype=torch.bool, device="cuda")
            if i == 0:
                hit[last:new[0], 2:] = True
            else:
                hit[last:new[0], 2:, 17] = True
            assert torch.equal(got[~hit], clean[~hit]), (new, i, hex(what))
            if what == 0x7FC0:
                assert torch.isnan(got[hit]).all()
            else:
                assert torch.isinf(got[hit]).all() and ((got[hit] > 0) == (what == 0x7F80)).all()


def test_attention_rows_of_lengths_that_do_not_fit(wq):
    # a length below the new tokens counts as equal to it; ranges that leave the rows are cut
    rng = np.random.default_rng(8)
    c = Cache(rng, [0], 2, 3, 64, 128, 128)
    q, kv = bf16_bits(rng, 5, 4, D), [bf16_bits(rng, 5, 2, D) for _ in range(2)]
    t = (dev16(q), dev16(kv[0]), dev16(kv[1]))
    a = wq.hlwq_kv_paged_attention(*t, i32([0, 5]), i32([5]), i32(c.table), *c.tensors())
    b = wq.hlwq_kv_paged_attention(*t, i32([0, 5]), i32([-3]), i32(c.table), *c.tensors())
    e = wq.hlwq_kv_paged_attention(*t, i32([-7, 2000]), i32([5]), i32(c.table), *c.tensors())
    f = torch.full_like(a, 3.0)
    wq.hlwq_kv_paged_attention(*t, i32([9, 2]), i32([5]), i32(c.table), *c.tensors(), out=f)
    assert torch.equal(a, b) and torch.equal(a, e) and bool((f == 3).all())


# ---------------------------------------------------------------------------
# prompts
# ---------------------------------------------------------------------------

def prompt_case(wq, seed, lens, q_heads, kv_heads, extra=0, pad=0, scale=1 / 16, sigma=1.0):
    rng = np.random.default_rng(seed)
    rows = sum(lens) + pad
    q = bf16_bits(rng, rows, q_heads, D, sigma=sigma)
    kv = [bf16_bits(rng, rows, kv_heads, D) for _ in range(2)]
    cu = np.concatenate([[0], np.cumsum(lens)])
    for x in (q, *kv):
        x[cu[-1]:] = 0x7FC0
    make = (lambda x: strided(x, extra)) if extra else dev16
    out = torch.full((rows, q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    wq.hlwq_prompt_attention(make(q), make(kv[0]), make(kv[1]), i32(cu), scale=scale, out=out)
    torch.cuda.synchronize()
    got = out.cpu().double().numpy()
    worst = 0
    for b, n in enumerate(lens):
        if n:
            r = slice(cu[b], cu[b + 1])
            k, v = (f64(x[r]).transpose(1, 0, 2) for x in kv)
            worst = max(worst, pr.check_attention(got[r], f64(q[r]), k, v, 0, 0, kv_heads, scale))
    assert np.all(got[cu[-1]:] == 7.0)
    print(f"largest error {worst:.3f} of its bound", flush=True)


@pytest.mark.parametrize("lens", [[1], [2], [15, 16, 17], [31, 32, 33], [63, 64, 65], [127], [129, 0, 1], [257], [0, 511, 0],
                                  [300, 5, 200], [1] * 40])
@pytest.mark.parametrize("q_heads,kv_heads", [(6, 1), (4, 2)])
def test_prompt_lengths(wq, lens, q_heads, kv_heads):
    prompt_case(wq, sum(lens), lens, q_heads, kv_heads)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (5, 5), (24, 4), (8, 1), (7, 1), (33, 1), (130, 1), (300, 1)])
def test_prompt_heads(wq, q_heads, kv_heads):
    prompt_case(wq, q_heads, [70, 3], q_heads, kv_heads, extra=16, pad=4)


def test_prompt_long(wq):
    prompt_case(wq, 1, [1500], 2, 1)


@pytest.mark.parametrize("scale,sigma", [(1 / 16, 8.0), (1.0, 0.01), (-0.05, 1.0), (0.0, 1.0), (1 / 16, 300.0)])
def test_prompt_scales(wq, scale, sigma):
    prompt_case(wq, 2, [200, 77], 6, 2, scale=scale, sigma=sigma)


def test_prompt_nan_and_infinities_stay_with_the_rows_that_see_them(wq):
    rng = np.random.default_rng(7)
    lens = [100, 90]
    q, kv = bf16_bits(rng, 190, 6, D), [bf16_bits(rng, 190, 2, D) for _ in range(2)]
    cu = i32([0, 100, 190])
    clean = wq.hlwq_prompt_attention(dev16(q), dev16(kv[0]), dev16(kv[1]), cu)
    for row, end in ((57, 100), (100, 190), (0, 100), (99, 100)):
        for i, what in ((0, 0x7FC0), (1, 0x7FC0), (1, 0x7F80), (1, 0xFF80)):
            dirty = [x.copy() for x in kv]
            dirty[i][row, 1, 200] = what
            got = wq.hlwq_prompt_attention(dev16(q), dev16(dirty[0]), dev16(dirty[1]), cu)
            hit = torch.zeros(190, 6, D, dtype=torch.bool, device="cuda")
            if i == 0:
                hit[row:end, 3:] = True
            else:
                hit[row:end, 3:, 200] = True
            assert torch.equal(got[~hit], clean[~hit]), (row, i, hex(what))
            if what == 0x7FC0:
                assert torch.isnan(got[hit]).all()
            else:
                assert torch.isinf(got[hit]).all() and ((got[hit] > 0) == (what == 0x7F80)).all()
    assert sum(lens) == 190


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

class Serving:
    """A serving loop's state on the device: the calls that a user's program makes, step by step."""

    def __init__(self, wq, slots, kv_heads, bits, page, residual, ring, pool, width):
        self.wq, self.kw = wq, dict(n_residual=residual, bits=bits)
        self.page, self.residual = page, residual
        self.tokens, self.n_free = i32([0] * slots), i32([pool])
        self.free, self.table = i32(np.arange(pool)), i32(np.full((slots, width), -1))
        self.cache = [torch.zeros(pool, kv_heads, page, 32 * bits, dtype=torch.uint8, device="cuda"),
                      torch.full((pool, kv_heads, page), float("nan"), dtype=torch.float16, device="cuda")]
        self.cache += [x.clone() for x in self.cache]
        self.cache += [torch.full((slots, kv_heads, ring, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                       for _ in range(2)]

    def step(self, q, k, v, n_new, reset=None):
        p = self.wq.hlwq_kv_page_plan(self.tokens, n_new, self.free, self.n_free, self.table, q.shape[0],
                                      page_size=self.page, n_residual=self.residual, reset=reset)
        out = self.wq.hlwq_kv_paged_attention(q, k, v, p.cu_new, p.lens, self.table, *self.cache, **self.kw)
        self.wq.hlwq_kv_paged_append(k, v, p.cu_new, p.lens, p.row_request, p.slots, *self.cache, **self.kw)
        return p, out


@pytest.mark.parametrize("bits,page,residual,ring", [(3, 16, 128, 128), (2, 64, 32, 40)])
def test_a_serving_loop(wq, bits, page, residual, ring):
    """Prompts, decode steps, drafted tokens and slot turnover, against the cache as the oracle keeps it."""
    rng = np.random.default_rng(bits)
    slots, hq, hk, width = 3, 6, 2, 40
    s = Serving(wq, slots, hk, bits, page, residual, ring, 60, width)
    history = [[[], []] for _ in range(slots)]  # bf16 keys and values of each slot's request
    for step, new in enumerate([[300, 40, 0], [1, 1, 150], [1, 1, 1], [4, 0, 1], [60, 2, 1], [1, 1, 1], [7, 200, 1]]):
        reset = [0, 0, 0] if step != 5 else [1, 0, 0]
        rows = sum(new) + step % 3
        q, k, v = (bf16_bits(rng, rows, h, D) for h in (hq, hk, hk))
        p, out = s.step(dev16(q), dev16(k), dev16(v), i32(new), torch.tensor(reset, dtype=torch.uint8).cuda())
        torch.cuda.synchronize()
        assert p.status.item() == 0
        got, cu = out.cpu().double().numpy(), np.concatenate([[0], np.cumsum(new)])
        whole = None
        if step == 0:  # nothing cached: the same as whole prompts
            whole = wq.hlwq_prompt_attention(dev16(q), dev16(k), dev16(v), p.cu_new).cpu().double().numpy()
        for b in range(slots):
            if reset[b]:
                history[b] = [[], []]
            r = slice(cu[b], cu[b + 1])
            held = len(history[b][0])
            enc = pr.encoded(held, residual)
            both = []
            for i, x in enumerate((k, v)):
                old = np.array(history[b][i][:enc], np.uint16).reshape(enc, hk, D)
                codes, n16 = pr.ref.kv_quantize_c(np.ascontiguousarray(old[None]), n_residual=0, bits=bits)
                far = pr.decoded(codes[0], n16[0].view(np.float16), bits) if enc else np.zeros((0, hk, D))
                near = np.array(history[b][i][enc:], np.uint16).reshape(-1, hk, D)
                both.append(np.concatenate([far, f64(near), f64(x[r])]).transpose(1, 0, 2))
                history[b][i].extend(x[r])
            if new[b]:
                pr.check_attention(got[r], f64(q[r]), *both, enc, held, hk)
                if whole is not None:
                    pr.check_attention(whole[r], f64(q[r]), *both, enc, held, hk)
        s.tokens, s.n_free = p.lens, p.n_free
    assert s.tokens.tolist() == [len(h[0]) for h in history]


def test_a_captured_step_replays(wq):
    """One decode step captured into a graph, replayed over new contents with eager work between, equals eager steps."""
    rng = np.random.default_rng(0)
    slots, hq, hk = 4, 12, 2
    make = lambda: Serving(wq, slots, hk, 3, 16, 128, 128, 120, 30)  # noqa: E731
    eager, graphed = make(), make()
    first = [dev16(bf16_bits(rng, 700, h, D)) for h in (hq, hk, hk)]
    for s in (eager, graphed):
        p, _ = s.step(*first, i32([130, 127, 40, 403]))
        s.tokens.copy_(p.lens)
        s.n_free.copy_(p.n_free)
    q, k, v = (torch.zeros(6, h, D, dtype=torch.bfloat16, device="cuda") for h in (hq, hk, hk))
    n_new = i32([0] * slots)

    def one(s):
        p, out = s.step(q, k, v, n_new)
        s.tokens.copy_(p.lens)
        s.n_free.copy_(p.n_free)
        return out

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        one(graphed)  # warm-up with no new tokens: changes nothing
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = one(graphed)
    for step in range(20):
        new = [1, int(step % 2), 1, 1] if step % 5 else [2, 1, 0, 3]
        for t, h in ((q, hq), (k, hk), (v, hk)):
            t.copy_(dev16(bf16_bits(rng, 6, h, D)))
        n_new.copy_(i32(new))
        want = one(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want[:sum(new)], held[:sum(new)]), step
        torch.rand(1 << 20, device="cuda").sum().item()
    for x, y in zip((eager.tokens, eager.n_free, eager.free, eager.table, *eager.cache),
                    (graphed.tokens, graphed.n_free, graphed.free, graphed.table, *graphed.cache)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_another_stream_and_two_calls_at_once(wq):
    rng = np.random.default_rng(2)
    ctx, new = [900, 300], [1, 1]
    c = [Cache(rng, ctx, 2, 3, 64, 128, 128) for _ in range(2)]
    q, k, v = (dev16(bf16_bits(rng, 2, h, D)) for h in (4, 2, 2))
    cu, lens = i32([0, 1, 2]), i32([901, 301])
    tables = [i32(x.table) for x in c]
    alone = [wq.hlwq_kv_paged_attention(q, k, v, cu, lens, t, *x.tensors()) for t, x in zip(tables, c)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [wq.hlwq_kv_paged_attention(q, k, v, cu, lens, t, *x.tensors(), stream=s)
               for t, x, s in zip(tables, c, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, g) for a, g in zip(alone, got))
    assert sum(new) == 2


def test_given_workspace_is_enough(wq):
    rng = np.random.default_rng(12)
    c = Cache(rng, [900, 300], 2, 3, 64, 128, 128)
    q, k, v = (dev16(bf16_bits(rng, 2, h, D)) for h in (4, 2, 2))
    args = (q, k, v, i32([0, 1, 2]), i32([901, 301]), i32(c.table), *c.tensors())
    want = wq.hlwq_kv_paged_attention(*args)
    need = wq.hlwq_kv_paged_attention_workspace(2, 2, 4, 2)
    guard = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    got = wq.hlwq_kv_paged_attention(*args, workspace=guard[:need])
    assert torch.equal(want, got) and bool((guard[need:] == 0xA5).all())
    with pytest.raises(wq.HLWQError):
        wq.hlwq_kv_paged_attention(*args, workspace=guard[:need - 16])


def test_python_refusals(wq):
    x = torch.zeros(4, 2, D, dtype=torch.bfloat16, device="cuda")
    cu = i32([0, 4])
    with pytest.raises(ValueError, match="do not divide"):
        wq.hlwq_prompt_attention(torch.zeros(4, 3, D, dtype=torch.bfloat16, device="cuda"), x, x, cu)
    with pytest.raises(ValueError, match="side by side"):
        wq.hlwq_prompt_attention(x.transpose(0, 1).contiguous().transpose(0, 1), x, x, cu)
    with pytest.raises(ValueError, match="rows"):
        wq.hlwq_prompt_attention(x, x[:3], x, cu)
    with pytest.raises(ValueError, match="out must"):
        wq.hlwq_prompt_attention(x, x, x, cu, out=x[:3].clone())
    with pytest.raises(TypeError, match="cu_seqlens"):
        wq.hlwq_prompt_attention(x, x, x, cu.long())
    with pytest.raises(wq.HLWQError):
        wq.hlwq_prompt_attention(x, x, x, cu, out=x)
