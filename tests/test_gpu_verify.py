"""GPU tests of the verification of drafted tokens against tests/verify_ref.py: every output is a whole number and equal."""
import numpy as np
import pytest

import verify_ref as vr

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import weight_quantization_amd as m
    m.load_library()
    return m


TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def trees(rng, counts, wide):
    parents = []
    for n in counts:
        parents += [-1 if i == 0 else max(0, i - 1 - int(rng.integers(0, wide))) for i in range(n)]
    return np.array(parents, np.int32)


def softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def inputs(rng, counts, wide, vocab, dtype, sampled, pad=0, sharp=2.0):
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(cu[-1]) + pad
    parents = np.concatenate([trees(rng, counts, wide), np.full(pad, -1, np.int32)])
    z = rng.standard_normal((rows, vocab)) * sharp
    p = torch.from_numpy(softmax(z)).to(TYPES[dtype])
    q = torch.from_numpy(softmax(z + rng.standard_normal((rows, vocab)))).to(TYPES[dtype])
    tokens = np.zeros(rows, np.int32)
    for b in range(len(counts)):
        for i in range(1, counts[b]):
            row = q[cu[b] + parents[cu[b] + i]].double().numpy()
            tokens[cu[b] + i] = rng.choice(vocab, p=row / row.sum()) if sampled else np.argsort(-row)[i % min(wide, vocab)]
    u, un = rng.random(rows).astype(np.float32), rng.random(len(counts)).astype(np.float32)
    return tokens, parents, cu, p, (q if sampled else None), u, un


def run(wq, tokens, parents, cu, p, q, u, un, **kw):
    t = [torch.from_numpy(np.asarray(x)).cuda() for x in (tokens, parents, cu)]
    v = wq.hlwq_verify_drafts(*t, p.cuda(), torch.from_numpy(u).cuda(), torch.from_numpy(un).cuda(),
                              draft=None if q is None else q.cuda(), **kw)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in v]


def check(wq, *x):
    got = run(wq, *x)
    tokens, parents, cu, p, q, u, un = x
    want = vr.verify(tokens, parents, cu, p.double().numpy(), None if q is None else q.double().numpy(), u, un)
    for name, a, b in zip(("n_kept", "next_token", "kept"), got, want):
        assert np.array_equal(a, b), (name, np.argwhere(a != b)[:5].tolist(), a[a != b][:5], b[a != b][:5])
    return want


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [1, 2, 3, 63, 64, 257, 1000, 4097, 32001])
def test_trees(wq, vocab, dtype, sampled):
    rng = np.random.default_rng(vocab)
    counts = [1, 0, 5, 9, 2, 30, 1, 0][:8 if vocab < 5000 else 6]
    check(wq, *inputs(rng, counts, 3, vocab, dtype, sampled, pad=vocab % 3))


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("wide", [1, 8, 200])
def test_long_trees_of_many_siblings(wq, wide, sampled):
    rng = np.random.default_rng(wide)
    check(wq, *inputs(rng, [200, 65, 64, 129, 300], wide, 50, "float32", sampled, sharp=0.3))


def test_probabilities_of_a_large_vocabulary(wq):
    rng = np.random.default_rng(1)
    check(wq, *inputs(rng, [4, 3, 4], 2, 300007, "float32", True))
    check(wq, *inputs(rng, [4, 3], 1, 300007, "bfloat16", False))


@pytest.mark.parametrize("sampled", [True, False])
def test_every_position_of_the_next_token(wq, sampled):
    # one row, u swept over the whole range, both ends among it
    rng = np.random.default_rng(2)
    vocab, n = 700, 400
    p = torch.from_numpy(np.repeat(softmax(rng.standard_normal((1, vocab))), n, 0)).float()
    p[:, 100:164] = 0
    u = np.linspace(0, 1, n, endpoint=False).astype(np.float32)
    u[-1] = np.float32(1 - 2.0 ** -24)
    x = (np.zeros(n, np.int32), np.full(n, -1, np.int32), np.arange(n + 1, dtype=np.int32), p, p if sampled else None,
         np.zeros(n, np.float32), u)
    _, nxt, _ = check(wq, *x)
    assert nxt[0] == 0 and nxt[-1] == vocab - 1 and not np.any((nxt >= 100) & (nxt < 164))


def test_a_draft_equal_to_the_target_is_kept_and_a_disjoint_one_is_not(wq):
    rng = np.random.default_rng(3)
    vocab, counts = 200, [6] * 50
    tokens, parents, cu, p, _, u, un = inputs(rng, counts, 1, vocab, "float32", True)
    tokens[1:] = [rng.choice(vocab, p=r / r.sum()) for r in p.double().numpy()[:-1]]
    n_kept, *_ = check(wq, tokens, parents, cu, p, p.clone(), u, un)
    assert np.all(n_kept == 6)
    half = p.clone()
    half[:, :100] = 0
    other = p.clone()
    other[:, 100:] = 0
    tokens[:] = rng.integers(0, 100, len(tokens))
    n_kept, nxt, _ = check(wq, tokens, parents, cu, half, other, u, un)
    assert np.all(n_kept == 1) and np.all(nxt >= 100)


def test_kept_tokens_are_distributed_as_the_targets(wq):
    # the first token after the root, over 40000 requests with three sampled siblings: chi square
    rng = np.random.default_rng(4)
    vocab, n = 12, 40000
    p1, q1 = softmax(rng.standard_normal(vocab) * 1.5), softmax(rng.standard_normal(vocab) * 1.5)
    rows = 4 * n
    cu = np.arange(0, rows + 1, 4, dtype=np.int32)
    parents = np.tile(np.array([-1, 0, 0, 0], np.int32), n)
    tokens = rng.choice(vocab, rows, p=q1).astype(np.int32)
    p, q = (torch.from_numpy(np.tile(x, (rows, 1))).float() for x in (p1, q1))
    n_kept, nxt, kept = run(wq, tokens, parents, cu, p, q, rng.random(rows).astype(np.float32), rng.random(n).astype(np.float32))
    first = np.where(n_kept > 1, tokens[np.maximum(kept[cu[:-1] + 1], 0)], nxt)
    got = np.bincount(first, minlength=vocab)
    chi = ((got - n * p1) ** 2 / (n * p1)).sum()
    assert chi < 11 + 6 * np.sqrt(22), chi  # mean 11, six standard deviations
    # the first sibling alone is kept with the overlap of both; six standard deviations
    assert (n_kept > 1).mean() > np.minimum(p1, q1).sum() - 3 / np.sqrt(n)


def test_values_out_of_range(wq):
    rng = np.random.default_rng(5)
    tokens, parents, cu, p, q, u, un = inputs(rng, [9, 9, 9], 2, 90, "float32", True, pad=4)
    tokens[3], tokens[12], tokens[20] = -1, 90, 2 ** 31 - 1
    parents[4], parents[13], parents[22], parents[1] = 4, 2 ** 31 - 1, -2 ** 31, 7
    check(wq, tokens, parents, cu, p, q, u, un)
    check(wq, tokens, parents, cu, p, None, u, un)
    # a prefix sum outside the rows: cut to them, nothing outside is touched
    wild = cu.copy()
    wild[1], wild[2] = 2 ** 31 - 1, -7
    got = run(wq, tokens, parents, wild, p, q, u, un)
    assert got[0].shape == (3,) and np.all(got[2] < len(tokens))


def test_rows_without_mass_and_with_nan(wq):
    p = torch.zeros(6, 70)
    p[2, 5] = 0.25                     # a row that does not sum to one
    p[3] = float("nan")
    p[4, 3], p[4, 60] = float("nan"), 0.5
    p[5, 9], p[5, 10] = -1.0, 1e-30
    n = 6
    x = (np.zeros(n, np.int32), np.full(n, -1, np.int32), np.arange(n + 1, dtype=np.int32), p, None, np.zeros(n, np.float32),
         np.full(n, 0.5, np.float32))
    _, nxt, _ = run(wq, *x)
    assert nxt.tolist() == [-1, -1, 5, -1, 60, 10]


def test_nodes_past_the_limit_are_passed_over(wq):
    rng = np.random.default_rng(6)
    n, vocab = 4200, 8
    tokens = rng.integers(0, vocab, n).astype(np.int32)
    parents = np.arange(-1, n - 1, dtype=np.int32)
    p = torch.from_numpy(softmax(rng.standard_normal((n, vocab)))).float()
    u = np.zeros(n, np.float32)  # everything is kept
    got = check(wq, tokens, parents, np.array([0, n], np.int32), p, p.clone(), u, np.array([0.3], np.float32))
    assert got[0][0] == 4096


@pytest.mark.parametrize("dtype,vocab", [("float32", 501), ("bfloat16", 1003), ("float16", 77)])
def test_strides_and_streams(wq, dtype, vocab):
    rng = np.random.default_rng(7)
    tokens, parents, cu, p, q, u, un = inputs(rng, [5, 7, 1], 2, vocab, dtype, True)
    want = run(wq, tokens, parents, cu, p, q, u, un)
    wide_p = torch.full((len(tokens), vocab + 13), float("nan"), dtype=TYPES[dtype], device="cuda")
    wide_q = torch.full((len(tokens), 2 * vocab + 1), float("nan"), dtype=TYPES[dtype], device="cuda")
    wide_p[:, 3:3 + vocab], wide_q[:, 1:1 + vocab] = p.cuda(), q.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t = [torch.from_numpy(x).cuda() for x in (tokens, parents, cu)]
    ud, und = torch.from_numpy(u).cuda(), torch.from_numpy(un).cuda()
    torch.cuda.synchronize()
    v = wq.hlwq_verify_drafts(*t, wide_p[:, 3:3 + vocab], ud, und, draft=wide_q[:, 1:1 + vocab], stream=s)
    s.synchronize()
    for a, b in zip(v, want):
        assert np.array_equal(a.cpu().numpy(), b)


def test_capture_and_replay(wq):
    rng = np.random.default_rng(8)
    counts = [6, 1, 9, 4]
    host = inputs(rng, counts, 3, 1234, "float32", True)
    d = [torch.from_numpy(np.asarray(x)).cuda() if not torch.is_tensor(x) else x.cuda() for x in host]
    tokens, parents, cu, p, q, u, un = d
    wq.hlwq_verify_drafts(tokens, parents, cu, p, u, un, draft=q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        v = wq.hlwq_verify_drafts(tokens, parents, cu, p, u, un, draft=q)
    for _ in range(4):
        u.copy_(torch.from_numpy(rng.random(u.shape[0]).astype(np.float32)))
        un.copy_(torch.from_numpy(rng.random(4).astype(np.float32)))
        want = wq.hlwq_verify_drafts(tokens, parents, cu, p, u, un, draft=q)
        for t in v:
            t.fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(v, want):
            assert torch.equal(a, b)


def test_no_requests_and_refusals(wq):
    z = torch.zeros
    i32 = dict(dtype=torch.int32, device="cuda")
    v = wq.hlwq_verify_drafts(z(0, **i32), z(0, **i32), z(1, **i32), z(0, 9, device="cuda"), z(0, device="cuda"), z(0, device="cuda"))
    assert all(x.numel() == 0 for x in v)
    v = wq.hlwq_verify_drafts(z(0, **i32), z(0, **i32), z(3, **i32), z(0, 9, device="cuda"), z(0, device="cuda"), z(2, device="cuda"))
    assert v.n_kept.tolist() == [0, 0] and v.next_token.tolist() == [-1, -1]
    p, u, un = z(4, 9, device="cuda"), z(4, device="cuda"), z(1, device="cuda")
    t, cu = z(4, **i32), z(2, **i32)
    with pytest.raises(TypeError):
        wq.hlwq_verify_drafts(t, t, cu, p.double(), u, un)
    with pytest.raises(TypeError):
        wq.hlwq_verify_drafts(t, t, cu, p, u, un, draft=p.half())
    with pytest.raises(ValueError):
        wq.hlwq_verify_drafts(t, t, cu, p, u, un, draft=p[:3])
    with pytest.raises(ValueError):
        wq.hlwq_verify_drafts(t, t, cu, p.t().contiguous().t(), u, un)
    with pytest.raises(ValueError):
        wq.hlwq_verify_drafts(t[:3], t, cu, p, u, un)
    with pytest.raises(ValueError):
        wq.hlwq_verify_drafts(t, t, cu, p[:, :0], u, un)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [70, 1003])
def test_a_draft_with_nan_and_negative_values(wq, vocab, dtype):
    """Probabilities below 0 and NaN count as 0, the draft's too: in the decisions and in the sums after refusals."""
    rng = np.random.default_rng(vocab)
    tokens, parents, cu, p, q, u, un = inputs(rng, [9, 40, 30, 50, 12, 5], 30, vocab, dtype, True)
    rows = np.repeat(cu[:-1], np.diff(cu)) + np.maximum(parents, 0)
    good = [t[rows, tokens].clone() for t in (p, q)]
    for t in (p, q):
        what = torch.from_numpy(rng.integers(0, 12, t.shape))
        t[what == 0] = float("nan")
        t[what == 1] = -t[what == 1]
    # a request's children as they were, most of them refused; of the others some kept over a q of 0
    most = np.arange(len(tokens)) < cu[4]
    for t, g in zip((p, q), good):
        t[rows[most], tokens[most]] = g[most]
    u[most] = 1 - 2.0 ** -10 * u[most]
    # a row of q that is nothing but NaN, and children that p does not have either
    q[0] = float("nan")
    p[0, tokens[1:cu[1]][parents[1:cu[1]] == 0]] = 0
    got = run(wq, tokens, parents, cu, p, q, u, un)
    clean = [torch.where(t > 0, t, 0).double().numpy() for t in (p, q)]
    want = vr.verify(tokens, parents, cu, *clean, u, un)
    assert want[0][0] == 1 and max(want[0]) > 1
    # children of a root that were refused before one was kept, or for good
    ends = [want[2][cu[b] + 1] if want[0][b] > 1 else cu[b + 1] for b in range(6)]
    assert sum(int(np.sum(parents[cu[b] + 1:ends[b]] == 0)) for b in range(1, 4)) > 2
    for name, a, b in zip(("n_kept", "next_token", "kept"), got, want):
        assert np.array_equal(a, b), (name, a, b)


@pytest.mark.parametrize("counts,before,pad", [([], 0, 5), ([], 3, 2000), ([2, 3], 4, 3), ([0, 1], 1500, 0)])
def test_rows_of_no_request_are_not_kept(wq, monkeypatch, counts, before, pad):
    rng = np.random.default_rng(before + pad)
    n, rows, vocab = len(counts), before + sum(counts) + pad, 40
    cu = (before + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    p = torch.from_numpy(softmax(rng.standard_normal((rows, vocab)))).float()
    tokens, parents = rng.integers(0, vocab, rows).astype(np.int32), np.full(rows, -1, np.int32)
    for b in range(n):
        parents[cu[b] + 1:cu[b + 1]] = np.arange(counts[b] - 1) if counts[b] else 0
    u, un = np.zeros(rows, np.float32), rng.random(n).astype(np.float32)  # everything is kept
    monkeypatch.setattr(wq.drafts, "_empty", lambda shape, dtype, device, stream: torch.full((shape,), 7, dtype=dtype, device=device))
    v = run(wq, tokens, parents, cu, p, None, u, un)
    own = slice(before, before + sum(counts))
    kept = np.full(rows, -1, np.int32)
    kept[own] = np.arange(rows)[own]
    assert np.array_equal(v[2], kept) and v[0].tolist() == counts
