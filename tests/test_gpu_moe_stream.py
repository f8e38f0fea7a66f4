"""GPU tests of the mixture-of-experts layer where many pairs meet large banks: banks streamed through LDS (160 blocks and
more of the down projections' rows among the touched experts, more than 32 pairs), and the same sizes in banks that lie so
that they are not."""
import numpy as np
import pytest

import moe_ref as mr
from test_gpu_moe import bank, bf16, dev, f64, wq  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def moved(t, by):
    """A tensor's values `by` bytes past an allocation's start."""
    raw = torch.empty(t.numel() * t.element_size() + by, dtype=torch.uint8, device="cuda")
    view = raw[by:].view(t.dtype).view(t.shape)
    view.copy_(t)
    return view


def given(wq, rng, tokens, experts, hidden, inner, k, bits, kind, among=None, put=dev):
    """A call with experts drawn from `among`, against the definition."""
    assert tokens * k > 32 and min(experts, tokens * k) * -(-inner // 128) >= 160
    x, xf = bf16(rng, tokens, hidden)
    up, down = bank(rng, experts, 2 * inner, hidden, bits), bank(rng, experts, hidden, inner, bits)
    ids = rng.choice(np.arange(experts) if among is None else among, (tokens, k)).astype(np.int32)
    w = rng.standard_normal((tokens, k)).astype(np.float32)
    y = wq.hlwq_moe_experts(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *put(up), *put(down), bits=bits,
                            activation=kind)
    worst = mr.check(f64(y), *mr.experts(xf, ids, w, up, down, bits, kind))
    print(f"largest error {worst:.3f} of its bound", flush=True)


@pytest.mark.parametrize("tokens,experts,hidden,inner,k", [
    (20, 160, 256, 128, 8), (170, 170, 128, 1, 1), (40, 128, 1, 130, 2), (40, 80, 300, 200, 8), (70, 43, 1000, 385, 8),
    (20, 160, 1150, 72, 8), (300, 18, 514, 1030, 4), (65, 3, 140, 7000, 1), (150, 3, 100, 8192, 1), (1000, 170, 260, 100, 6),
    (34, 15, 2050, 1300, 1), (64, 256, 640, 96, 32),
])
@pytest.mark.parametrize("bits,kind", [(5, "silu"), (3, "gelu_tanh")])
def test_sizes(wq, tokens, experts, hidden, inner, k, bits, kind):
    given(wq, np.random.default_rng(tokens * 100 + inner), tokens, experts, hidden, inner, k, bits, kind)


@pytest.mark.parametrize("bits", [5, 3])
def test_the_widest_rows(wq, bits):
    # 192 blocks of a token's activations; few of many experts named
    given(wq, np.random.default_rng(1), 41, 160, 24500, 20, 4, bits, "silu", among=[0, 77, 127])


@pytest.mark.parametrize("bits,kind", [(5, "gelu_tanh"), (3, "silu")])
@pytest.mark.parametrize("among", [[5], [0, 129], [-1, 130, 2 ** 31 - 1, -2 ** 31, 64], [7, 8, 9, -1]])
def test_uneven_routings(wq, bits, kind, among):
    # one expert's pairs are more than a pass holds; experts out of range; the same expert twice for a token
    given(wq, np.random.default_rng(2), 100, 130, 400, 150, 3, bits, kind, among=among)


@pytest.mark.parametrize("bits", [5, 3])
@pytest.mark.parametrize("by", [4, 8])
def test_banks_that_lie_otherwise(wq, bits, by):
    given(wq, np.random.default_rng(3), 40, 80, 300, 200, 4, bits, "silu", put=lambda b: [moved(t, by) for t in dev(b)])


def test_norms_at_odd_places(wq):
    given(wq, np.random.default_rng(4), 40, 80, 300, 200, 4, 5, "silu", put=lambda b: [moved(t, i * 2) for i, t in enumerate(dev(b))])
    # an odd number of norms to an expert
    given(wq, np.random.default_rng(5), 40, 55, 301, 300, 4, 5, "silu")


def test_inner_sizes_past_what_streams(wq):
    given(wq, np.random.default_rng(6), 34, 3, 130, 8193, 1, 3, "silu")


@pytest.mark.parametrize("tokens,experts,hidden,inner,k", [(32, 300, 256, 200, 1), (2, 700, 300, 64, 16), (1, 1024, 8192, 10, 32),
                                                            (1, 1024, 8193, 130, 32), (33, 400, 129, 8, 1)])
@pytest.mark.parametrize("bits", [5, 3])
def test_about_thirty_two_pairs(wq, tokens, experts, hidden, inner, k, bits):
    rng = np.random.default_rng(tokens + hidden)
    x, xf = bf16(rng, tokens, hidden)
    router, rf = bf16(rng, experts, hidden, sigma=1.5 / np.sqrt(hidden))
    up, down = bank(rng, experts, 2 * inner, hidden, bits), bank(rng, experts, hidden, inner, bits)
    y = wq.hlwq_moe_layer(x.cuda(), router.cuda(), *dev(up), *dev(down), top_k=k, bits=bits)
    ids, w = mr.route(xf, rf, k, True)
    assert np.array_equal(y.experts.cpu().numpy(), ids)
    assert np.all(np.abs(y.weights.cpu().numpy() - w) <= 2.0 ** -24 * w + 1e-14)
    mr.check(f64(y.out), *mr.experts(xf, ids, y.weights.cpu().numpy(), up, down, bits, "silu"))


@pytest.mark.parametrize("tokens,experts,hidden,inner,k", [(16, 8, 1024, 520, 2), (4, 40, 2048, 512, 8), (2, 40, 2048, 512, 8),
                                                            (16, 64, 512, 256, 4), (40, 64, 300, 200, 8), (64, 8, 512, 500, 2)])
@pytest.mark.parametrize("bits", [5, 3])
def test_either_side_of_what_streams(wq, tokens, experts, hidden, inner, k, bits):
    """Fewer sets of rows than the streaming asks for, and pairs that are few or not by what they read."""
    rng = np.random.default_rng(tokens + inner)
    x, xf = bf16(rng, tokens, hidden)
    up, down = bank(rng, experts, 2 * inner, hidden, bits), bank(rng, experts, hidden, inner, bits)
    ids, w = rng.integers(0, experts, (tokens, k)).astype(np.int32), rng.standard_normal((tokens, k)).astype(np.float32)
    y = wq.hlwq_moe_experts(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *dev(up), *dev(down), bits=bits)
    mr.check(f64(y), *mr.experts(xf, ids, w, up, down, bits, "silu"))


@pytest.mark.parametrize("bits", [5, 3])
def test_a_bad_row_stays_in_its_row(wq, bits):
    rng = np.random.default_rng(7)
    tokens, experts, hidden, inner = 80, 128, 300, 150
    x, _ = bf16(rng, tokens, hidden)
    up, down = dev(bank(rng, experts, 2 * inner, hidden, bits)), dev(bank(rng, experts, hidden, inner, bits))
    ids = torch.tensor([[0, 2]] * tokens, dtype=torch.int32, device="cuda")
    w = torch.rand(tokens, 2, device="cuda")
    good = wq.hlwq_moe_experts(x.cuda(), ids, w, *up, *down, bits=bits)
    bad = x.clone()
    bad[0, 5], bad[1, 299], bad[40, 0] = float("nan"), float("inf"), float("-inf")
    y = wq.hlwq_moe_experts(bad.cuda(), ids, w, *up, *down, bits=bits)
    rows = torch.tensor([0, 1, 40], device="cuda")
    others = torch.ones(tokens, dtype=torch.bool, device="cuda").index_fill(0, rows, False)
    assert torch.isnan(y[rows]).all() and torch.equal(y[others], good[others])


@pytest.mark.parametrize("sigma", [1e-30, 1e17])
def test_small_and_large_activations(wq, sigma):
    rng = np.random.default_rng(8)
    experts, hidden, inner = 160, 256, 100
    x, xf = bf16(rng, 40, hidden, sigma=sigma)
    up, down = bank(rng, experts, 2 * inner, hidden, 5), bank(rng, experts, hidden, inner, 5)
    ids, w = rng.integers(0, experts, (40, 4)).astype(np.int32), rng.random((40, 4)).astype(np.float32)
    y = wq.hlwq_moe_experts(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *dev(up), *dev(down))
    ref, bound = mr.experts(xf, ids, w, up, down, 5, "silu")
    # (values under fp32's smallest normal number, 2^-126, keep what is left of them)
    mr.check(f64(y), ref, bound + 2.0 ** -126)


@pytest.mark.parametrize("tokens,bits", [(40, 5), (200, 3), (700, 5)])
def test_replays_streams_and_repeats(wq, tokens, bits):
    """Captured calls, two at once on streams of their own, the same bits each time, and nothing past the workspace."""
    rng = np.random.default_rng(9)
    experts, hidden, inner, k = 64, 520, 260, 8
    router = bf16(rng, experts, hidden)[0].cuda()
    up, down = dev(bank(rng, experts, 2 * inner, hidden, bits)), dev(bank(rng, experts, hidden, inner, bits))
    x = bf16(rng, tokens, hidden)[0].cuda()
    size = wq.hlwq_moe_workspace(experts, hidden, inner, tokens, k)
    ws = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    call = lambda **kw: wq.hlwq_moe_layer(x, router, *up, *down, top_k=k, bits=bits, **kw)
    want = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [ws[:size], torch.full((size,), 255, dtype=torch.uint8, device="cuda")]
    torch.cuda.synchronize()
    ys = [call(workspace=spaces[i % 2], stream=streams[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    for y in ys:
        assert all(torch.equal(a, b) for a, b in zip(y, want))
    assert bool((ws[size:] == 255).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = call(workspace=ws)
    for _ in range(4):
        x.copy_(bf16(rng, tokens, hidden)[0])
        want = call()
        for t in y:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(y, want))


def test_two_graphs_share_a_workspace(wq):
    """Captured calls of different sizes, kernels and bits on one workspace, replayed in turn between eager calls on it."""
    rng = np.random.default_rng(10)
    experts, hidden, inner, k = 64, 520, 260, 8
    router = bf16(rng, experts, hidden)[0].cuda()
    banks = {b: (*dev(bank(rng, experts, 2 * inner, hidden, b)), *dev(bank(rng, experts, hidden, inner, b))) for b in (5, 3)}
    xs = [bf16(rng, n, hidden)[0].cuda() for n in (40, 1, 7)]
    ws = torch.empty(wq.hlwq_moe_workspace(experts, hidden, inner, 40, k), dtype=torch.uint8, device="cuda")
    call = lambda i, **kw: wq.hlwq_moe_layer(xs[i], router, *banks[3 if i == 2 else 5], top_k=k, bits=3 if i == 2 else 5, **kw)
    graphs, outs = [], []
    for i in range(3):
        call(i, workspace=ws)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(call(i, workspace=ws))
    for _ in range(3):
        for x in xs:
            x.copy_(bf16(rng, *x.shape)[0])
        wants = [call(i) for i in range(3)]
        for i in (1, 0, 2, 0, 1):
            for t in outs[i]:
                t.zero_()
            graphs[i].replay()
            assert all(torch.equal(a, b) for a, b in zip(outs[i], wants[i]))
            ws.fill_(255)


@pytest.mark.parametrize("tokens,experts,hidden,inner,k", [
    # several passes over one bank or both, few enough to be streamed ..
    (40, 20, 140, 7000, 1), (60, 20, 140, 7000, 2), (80, 20, 100, 8192, 2), (100, 16, 2100, 1270, 4), (70, 80, 5120, 130, 4),
    # .. and too many
    (200, 80, 5120, 130, 8), (150, 24, 8200, 840, 5), (130, 3, 130, 8190, 2),
])
@pytest.mark.parametrize("bits", [5, 3])
def test_either_side_of_what_passes_cost(wq, tokens, experts, hidden, inner, k, bits):
    given(wq, np.random.default_rng(tokens + hidden), tokens, experts, hidden, inner, k, bits, "silu")


@pytest.mark.parametrize("tokens,experts,hidden,inner,k", [
    # one token's pairs, up to eight, and inner values of up to 16 blocks ..
    (1, 9, 4000, 2048, 8), (1, 9, 4000, 2048, 9), (1, 5, 300, 2049, 2), (2, 9, 4000, 700, 4),
    # .. and 393216 blocks in all
    (32, 40, 1024, 256, 1), (8, 20, 2048, 256, 4), (8, 20, 2048, 257, 4),
])
@pytest.mark.parametrize("bits", [5, 3])
def test_either_side_of_what_is_little(wq, tokens, experts, hidden, inner, k, bits):
    rng = np.random.default_rng(hidden + inner)
    x, xf = bf16(rng, tokens, hidden)
    router, rf = bf16(rng, experts, hidden, sigma=1.5 / np.sqrt(hidden))
    up, down = bank(rng, experts, 2 * inner, hidden, bits), bank(rng, experts, hidden, inner, bits)
    y = wq.hlwq_moe_layer(x.cuda(), router.cuda(), *dev(up), *dev(down), top_k=k, bits=bits)
    ids, _ = mr.route(xf, rf, k, True)
    assert np.array_equal(y.experts.cpu().numpy(), ids)
    mr.check(f64(y.out), *mr.experts(xf, ids, y.weights.cpu().numpy(), up, down, bits, "silu"))
