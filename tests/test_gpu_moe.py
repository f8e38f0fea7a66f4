"""GPU tests of the mixture-of-experts layer against its definition in 64 bits (tests/moe_ref.py)."""
import numpy as np
import pytest

import moe_ref as mr

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import weight_quantization_amd as m
    m.load_library()
    return m


def bank(rng, experts, out, n_in, bits):
    nb = -(-n_in // 128)
    packed = rng.integers(0, 256, (experts, out, nb, 16 * bits), dtype=np.uint8)
    norms = (0.2 + 0.1 * rng.standard_normal((experts, out, nb))).clip(0.01).astype(np.float16)
    return packed, norms


def bf16(rng, *shape, sigma=1.0):
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(sigma)).to(torch.bfloat16)
    return t, t.float().numpy()


def dev(b):
    return tuple(torch.from_numpy(x).cuda() for x in b)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


SIZES = [
    # tokens, experts, hidden, inner, top_k, bits, activation
    (1, 8, 256, 128, 2, 5, "silu"), (1, 256, 128, 128, 8, 3, "silu"), (2, 5, 129, 127, 1, 5, "gelu_tanh"),
    (3, 7, 1, 1, 3, 3, "silu"), (7, 64, 1000, 200, 8, 5, "gelu_tanh"), (16, 4, 384, 96, 2, 3, "gelu_tanh"),
    (17, 3, 640, 72, 3, 5, "silu"), (33, 2, 130, 260, 1, 3, "silu"), (65, 6, 700, 900, 4, 5, "silu"),
    (19, 11, 2816, 704, 2, 5, "gelu_tanh"), (5, 9, 5120, 136, 2, 3, "silu"), (4, 4, 300, 1500, 4, 5, "silu"),
    (2, 1024, 160, 16, 32, 3, "silu"), (9, 300, 200, 40, 10, 5, "silu"), (5, 1, 256, 256, 1, 5, "silu"),
]


@pytest.mark.parametrize("tokens,experts,hidden,inner,top_k,bits,kind", SIZES)
def test_layer(wq, tokens, experts, hidden, inner, top_k, bits, kind):
    rng = np.random.default_rng(tokens * 1000 + hidden)
    x, xf = bf16(rng, tokens, hidden)
    router, rf = bf16(rng, experts, hidden, sigma=1.5 / np.sqrt(hidden))
    up, down = bank(rng, experts, 2 * inner, hidden, bits), bank(rng, experts, hidden, inner, bits)
    renorm = bool(tokens % 2)
    y = wq.hlwq_moe_layer(x.cuda(), router.cuda(), *dev(up), *dev(down), top_k=top_k, bits=bits, activation=kind,
                          renormalize=renorm)
    ids, w = mr.route(xf, rf, top_k, renorm)
    assert np.array_equal(y.experts.cpu().numpy(), ids)
    # one rounding to fp32 of 64-bit values
    assert np.all(np.abs(y.weights.cpu().numpy() - w) <= 2.0 ** -24 * w + 1e-14)
    ref, bound = mr.experts(xf, ids, y.weights.cpu().numpy(), up, down, bits, kind)
    mr.check(f64(y.out), ref, bound)
    # the same routing given
    z = wq.hlwq_moe_experts(x.cuda(), y.experts, y.weights, *dev(up), *dev(down), bits=bits, activation=kind)
    assert torch.equal(z, y.out)


def test_many_tokens_take_several_passes(wq):
    rng = np.random.default_rng(3)
    tokens, experts, hidden, inner, k = 1111, 9, 150, 140, 8
    x, xf = bf16(rng, tokens, hidden)
    up, down = bank(rng, experts, 2 * inner, hidden, 5), bank(rng, experts, hidden, inner, 5)
    ids = rng.integers(0, experts, (tokens, k)).astype(np.int32)
    w = rng.random((tokens, k)).astype(np.float32)
    y = wq.hlwq_moe_experts(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *dev(up), *dev(down))
    mr.check(f64(y), *mr.experts(xf, ids, w, up, down, 5, "silu"))


def test_layer_of_several_passes(wq):
    rng = np.random.default_rng(4)
    tokens, experts, hidden, inner, k = 300, 40, 130, 20, 32
    x, xf = bf16(rng, tokens, hidden)
    router, rf = bf16(rng, experts, hidden, sigma=0.1)
    up, down = bank(rng, experts, 2 * inner, hidden, 3), bank(rng, experts, hidden, inner, 3)
    y = wq.hlwq_moe_layer(x.cuda(), router.cuda(), *dev(up), *dev(down), top_k=k, bits=3)
    ids, w = mr.route(xf, rf, k, True)
    assert np.array_equal(y.experts.cpu().numpy(), ids)
    mr.check(f64(y.out), *mr.experts(xf, ids, y.weights.cpu().numpy(), up, down, 3, "silu"))


@pytest.mark.parametrize("tokens", [1, 3, 40])
def test_equal_logits_go_to_the_lowest_index(wq, tokens):
    rng = np.random.default_rng(tokens)
    x, xf = bf16(rng, tokens, 200)
    router, rf = bf16(rng, 12, 200)
    router, rf = router[[0, 1, 1, 0, 2, 2, 0, 1, 3, 3, 3, 0]], rf[[0, 1, 1, 0, 2, 2, 0, 1, 3, 3, 3, 0]]
    up, down = bank(rng, 12, 64, 200, 5), bank(rng, 12, 200, 32, 5)
    y = wq.hlwq_moe_layer(x.cuda(), router.contiguous().cuda(), *dev(up), *dev(down), top_k=5)
    assert np.array_equal(y.experts.cpu().numpy(), mr.route(xf, rf, 5, True)[0])
    zero = wq.hlwq_moe_layer(torch.zeros_like(x).cuda(), router.contiguous().cuda(), *dev(up), *dev(down), top_k=5)
    assert torch.equal(zero.experts.cpu(), torch.arange(5, dtype=torch.int32).expand(tokens, 5))
    assert torch.all(zero.out == 0)


def test_logits_that_fp32_does_not_tell_apart(wq):
    # expert 1 leads expert 0 by 2^-14 in sums around 2^12: beyond fp32
    x = torch.ones(3, 256, dtype=torch.bfloat16)
    router = torch.full((4, 256), 16.0, dtype=torch.bfloat16)
    router[2:] = -1
    router[1, 7] = 16.0
    x[:, 7] = 2.0 ** -20
    router[1, 7], router[0, 7] = 64.0, 0.0
    rng = np.random.default_rng(0)
    up, down = bank(rng, 4, 32, 256, 5), bank(rng, 4, 256, 16, 5)
    y = wq.hlwq_moe_layer(x.cuda(), router.cuda(), *dev(up), *dev(down), top_k=2)
    assert torch.equal(y.experts.cpu(), torch.tensor([[1, 0]] * 3, dtype=torch.int32))


@pytest.mark.parametrize("tokens", [1, 6, 40])
def test_experts_out_of_range_and_named_twice(wq, tokens):
    rng = np.random.default_rng(11)
    experts, hidden, inner, k = 6, 260, 140, 4
    x, xf = bf16(rng, tokens, hidden)
    up, down = bank(rng, experts, 2 * inner, hidden, 5), bank(rng, experts, hidden, inner, 5)
    ids = rng.integers(0, experts, (tokens, k)).astype(np.int32)
    ids[0] = [2, 2, -1, 6]
    ids[-1] = [-2 ** 31, 2 ** 31 - 1, -1, 1024] if tokens > 1 else ids[-1]
    w = rng.standard_normal((tokens, k)).astype(np.float32)
    y = wq.hlwq_moe_experts(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *dev(up), *dev(down),
                            activation="gelu_tanh")
    mr.check(f64(y), *mr.experts(xf, ids, w, up, down, 5, "gelu_tanh"))
    if tokens > 1:
        assert torch.all(y[-1] == 0)


@pytest.mark.parametrize("tokens", [3, 33])
def test_a_bad_row_stays_in_its_row(wq, tokens):
    rng = np.random.default_rng(5)
    experts, hidden, inner = 4, 300, 150
    x, xf = bf16(rng, tokens, hidden)
    up, down = bank(rng, experts, 2 * inner, hidden, 5), bank(rng, experts, hidden, inner, 5)
    ids = np.tile(np.array([[0, 2]], np.int32), (tokens, 1))
    w = rng.random((tokens, 2)).astype(np.float32)
    good = wq.hlwq_moe_experts(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *dev(up), *dev(down))
    bad = x.clone()
    bad[0, 5], bad[1, 299] = float("nan"), float("inf")
    y = wq.hlwq_moe_experts(bad.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *dev(up), *dev(down))
    assert torch.isnan(y[:2]).all() and torch.equal(y[2:], good[2:])


@pytest.mark.parametrize("sigma", [1e-30, 1e-12, 1e12, 1e17])
def test_small_and_large_activations(wq, sigma):
    rng = np.random.default_rng(6)
    experts, hidden, inner = 3, 256, 200
    x, xf = bf16(rng, 4, hidden, sigma=sigma)
    up, down = bank(rng, experts, 2 * inner, hidden, 5), bank(rng, experts, hidden, inner, 5)
    ids = np.tile(np.array([[0, 2]], np.int32), (4, 1))
    w = rng.random((4, 2)).astype(np.float32)
    y = wq.hlwq_moe_experts(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *dev(up), *dev(down))
    ref, bound = mr.experts(xf, ids, w, up, down, 5, "silu")
    # (values under fp32's smallest normal number, 2^-126, keep what is left of them)
    mr.check(f64(y), ref, bound + 2.0 ** -126)


def test_strides_streams_workspace_and_edges(wq):
    rng = np.random.default_rng(8)
    experts, hidden, inner, k = 5, 200, 90, 2
    x, xf = bf16(rng, 9, hidden)
    router, _ = bf16(rng, experts, hidden)
    up, down = dev(bank(rng, experts, 2 * inner, hidden, 5)), dev(bank(rng, experts, hidden, inner, 5))
    router = router.cuda()
    want = wq.hlwq_moe_layer(x.cuda(), router, *up, *down, top_k=k)
    wide = torch.full((9, 3 * hidden + 1), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 7:7 + hidden] = x.cuda()
    size = wq.hlwq_moe_workspace(experts, hidden, inner, 9, k)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((9, hidden), float("nan"), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = wq.hlwq_moe_layer(wide[:, 7:7 + hidden], router, *up, *down, top_k=k, out=out, workspace=ws, stream=s)
    s.synchronize()
    assert y.out is out
    for a, b in zip(y, want):
        assert torch.equal(a, b)
    # nothing past the workspace that was asked for
    big = torch.full((size + 4096,), 7, dtype=torch.uint8, device="cuda")
    wq.hlwq_moe_layer(x.cuda(), router, *up, *down, top_k=k, workspace=big[:size])
    assert torch.all(big[size:] == 7)
    assert wq.hlwq_moe_layer(x[:0].cuda(), router, *up, *down, top_k=k).out.shape == (0, hidden)
    none = wq.hlwq_moe_layer(x.cuda(), router, *up, *down, top_k=0)
    assert torch.all(none.out == 0) and none.experts.shape == (9, 0)
    flat = torch.empty(9, 0, dtype=torch.bfloat16, device="cuda")
    up0, down0 = bank(rng, experts, 2 * inner, 0, 5), bank(rng, experts, 0, inner, 5)
    assert wq.hlwq_moe_layer(flat, router[:, :0].contiguous(), *dev(up0), *dev(down0), top_k=k).out.shape == (9, 0)
    up0, down0 = bank(rng, experts, 0, hidden, 5), bank(rng, experts, hidden, 0, 5)
    assert torch.all(wq.hlwq_moe_layer(x.cuda(), router, *dev(up0), *dev(down0), top_k=k).out == 0)


@pytest.mark.parametrize("tokens", [1, 4, 50])
def test_capture_and_replay(wq, tokens):
    rng = np.random.default_rng(9)
    experts, hidden, inner, k = 16, 512, 256, 4
    router = bf16(rng, experts, hidden)[0].cuda()
    up, down = dev(bank(rng, experts, 2 * inner, hidden, 5)), dev(bank(rng, experts, hidden, inner, 5))
    x = bf16(rng, tokens, hidden)[0].cuda()
    ws = torch.empty(wq.hlwq_moe_workspace(experts, hidden, inner, tokens, k), dtype=torch.uint8, device="cuda")
    wq.hlwq_moe_layer(x, router, *up, *down, top_k=k, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = wq.hlwq_moe_layer(x, router, *up, *down, top_k=k, workspace=ws)
    for _ in range(4):
        x.copy_(bf16(rng, tokens, hidden)[0])
        want = wq.hlwq_moe_layer(x, router, *up, *down, top_k=k)
        for t in y:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(y, want):
            assert torch.equal(a, b)


def test_results_repeat_bit_for_bit(wq):
    rng = np.random.default_rng(10)
    experts, hidden, inner, k = 32, 640, 300, 8
    x, router = bf16(rng, 70, hidden)[0].cuda(), bf16(rng, experts, hidden)[0].cuda()
    up, down = dev(bank(rng, experts, 2 * inner, hidden, 5)), dev(bank(rng, experts, hidden, inner, 5))
    first = wq.hlwq_moe_layer(x, router, *up, *down, top_k=k)
    for _ in range(5):
        assert torch.equal(wq.hlwq_moe_layer(x, router, *up, *down, top_k=k).out, first.out)


def test_a_quantized_bank(wq):
    # hlwq_quantize's own output, against the products of its dequantized weights
    rng = np.random.default_rng(12)
    experts, hidden, inner, k = 4, 512, 320, 2
    up = (torch.from_numpy(rng.standard_normal((experts, 2 * inner, hidden)).astype(np.float32)) * 0.02).to(torch.bfloat16).cuda()
    down = (torch.from_numpy(rng.standard_normal((experts, hidden, inner)).astype(np.float32)) * 0.02).to(torch.bfloat16).cuda()
    qu, qd = wq.hlwq_quantize(up), wq.hlwq_quantize(down)
    x, router = bf16(rng, 6, hidden)[0].cuda(), bf16(rng, experts, hidden)[0].cuda()
    y = wq.hlwq_moe_layer(x, router, *qu, *qd, top_k=k)
    wu = wq.hlwq_dequantize(*qu, hidden).double()
    wd = wq.hlwq_dequantize(*qd, inner).double()
    ref = torch.zeros(6, hidden, dtype=torch.float64, device="cuda")
    for t in range(6):
        for e, w in zip(y.experts[t].tolist(), y.weights[t].tolist()):
            a = wu[e] @ x[t].double()
            h = torch.nn.functional.silu(a[:inner]) * a[inner:]
            ref[t] += w * (wd[e] @ h)
    # weights rounded to bf16 (2^-8) in the reference alone, over sums of hundreds of terms of either sign
    assert float((y.out.double() - ref).norm() / ref.norm()) < 2.0 ** -6


def test_refusals_raise(wq):
    rng = np.random.default_rng(13)
    up, down = dev(bank(rng, 4, 64, 256, 5)), dev(bank(rng, 4, 256, 32, 5))
    x, router = bf16(rng, 2, 256)[0].cuda(), bf16(rng, 4, 256)[0].cuda()
    with pytest.raises(ValueError):
        wq.hlwq_moe_layer(x, router, *up, *down, top_k=5)
    with pytest.raises(ValueError):
        wq.hlwq_moe_layer(x, router, *up, *down, top_k=2, bits=3)
    with pytest.raises(ValueError):
        wq.hlwq_moe_layer(x, router, *up, *down, top_k=2, activation="relu")
    with pytest.raises(ValueError):
        wq.hlwq_moe_layer(x.t(), router, *up, *down, top_k=2)
    with pytest.raises(TypeError):
        wq.hlwq_moe_layer(x.float(), router, *up, *down, top_k=2)
    with pytest.raises(wq.HLWQError):
        wq.hlwq_moe_layer(x, router, *up, *down, top_k=2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(wq.HLWQError):
        wq.hlwq_moe_layer(x, router, *up, *down, top_k=2, out=x)


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (3, 7, 7), (200, 300, 5)])
def test_rows_of_nothing_are_routed_all_the_same(wq, monkeypatch, tokens, experts, k, renormalize):
    """No hidden values: every logit is 0, so the first experts are chosen, with equal weights."""
    empty = torch.empty
    monkeypatch.setattr(wq.moe, "_empty", lambda shape, dtype, device, stream: empty(shape, dtype=dtype, device=device).fill_(77))
    rng = np.random.default_rng(0)
    up, down = bank(rng, experts, 64, 0, 5), bank(rng, experts, 0, 32, 5)
    x, router = (torch.zeros(n, 0, dtype=torch.bfloat16, device="cuda") for n in (tokens, experts))
    y = wq.hlwq_moe_layer(x, router, *dev(up), *dev(down), top_k=k, renormalize=renormalize)
    assert y.out.shape == (tokens, 0)
    assert torch.equal(y.experts.cpu(), torch.arange(k, dtype=torch.int32).expand(tokens, k))
    assert np.array_equal(y.weights.cpu().numpy(), np.full((tokens, k), np.float32(1 / (k if renormalize else experts))))


def test_row_strides_up_to_the_limit(wq):
    # a token of each of two sequences of 512 x 2048: rows 2^20 elements apart, and of 513 x 2048, which is refused
    rng = np.random.default_rng(14)
    up, down = dev(bank(rng, 4, 64, 2048, 5)), dev(bank(rng, 4, 2048, 32, 5))
    x, router = bf16(rng, 2, 2048)[0].cuda(), bf16(rng, 4, 2048)[0].cuda()
    want = wq.hlwq_moe_layer(x, router, *up, *down, top_k=2)
    h = torch.zeros(2, 513, 2048, dtype=torch.bfloat16, device="cuda")
    h[:, -1] = x
    near = h.view(-1)[:2 * 512 * 2048].view(2, 512, 2048)
    near[:, -1] = x
    assert near[:, -1].stride() == (2 ** 20, 1)
    assert all(torch.equal(a, b) for a, b in zip(wq.hlwq_moe_layer(near[:, -1], router, *up, *down, top_k=2), want))
    h[:, -1] = x
    with pytest.raises(wq.HLWQError):
        wq.hlwq_moe_layer(h[:, -1], router, *up, *down, top_k=2)
    assert torch.equal(wq.hlwq_moe_layer(h[:, -1].contiguous(), router, *up, *down, top_k=2).out, want.out)
    assert torch.equal(wq.hlwq_moe_layer(h[1:, -1], router, *up, *down, top_k=2).out, want.out[1:])  # there is no next row
