"""Sizes whose element offsets pass 32 bits: the last rows against the same rows computed alone."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_moe_expert_sort_amd as m
    m.lib()
    return m, torch.device("cuda:0")


def test_select_past_32_bits(gpu):
    import torch
    m, dev = gpu
    T, E = (1 << 24) + 5, 256  # 2^32 + 1280 logits
    l = torch.empty(T, E, dtype=torch.bfloat16, device=dev)
    block = torch.randn(1 << 20, E, device=dev).to(torch.bfloat16)
    for t in range(0, T, 1 << 20):
        l[t:t + (1 << 20)] = block[:min(1 << 20, T - t)]
    ids, probs = m.router_select(l, 8)
    a, b = m.router_select(l[-37:].contiguous(), 8)
    assert torch.equal(ids[-37:], a) and torch.equal(probs[-37:], b)
    dp = torch.ones_like(probs)
    dp[:, 0] = 2.0
    g = m.router_select_backward(l, ids, dp, renormalize=False)
    assert torch.equal(g[-37:], m.router_select_backward(l[-37:].contiguous(), a, dp[-37:].contiguous(), renormalize=False))


def test_mxfp4_past_32_bits(gpu):
    import torch
    m, dev = gpu
    rows, cols = 70001, 65536  # 4.6e9 elements
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
    block = torch.randn(4096, cols, device=dev).to(torch.bfloat16)
    for r in range(0, rows, 4096):
        x[r:r + 4096] = block[:min(4096, rows - r)]
    codes, scales = m.mxfp4_quantize(x)
    a, b = m.mxfp4_quantize(x[-9:].contiguous())
    assert torch.equal(codes[-9:], a) and torch.equal(scales[-9:], b)
    assert torch.equal(m.mxfp4_dequantize(codes, scales)[-9:], m.mxfp4_dequantize(a, b))


def test_linear_past_32_bits(gpu):
    import torch
    m, dev = gpu
    M, N, K = 70001, 65600, 64  # 4.6e9 outputs
    w = m.Mxfp4Weights(1, N, K, dev).quantize_from(torch.randn(1, N, K, device=dev).to(torch.bfloat16))
    x = torch.randn(M, K, device=dev).to(torch.bfloat16)
    y = m.mxfp4_linear(x, w)
    for r in (0, 40000, M - 5):
        assert torch.equal(y[r:r + 5], m.mxfp4_linear(x[r:r + 5].contiguous(), w))


def test_grouped_weights_past_32_bits(gpu):
    """Weights of more than 4 GiB of codes: the last experts."""
    import torch
    m, dev = gpu
    E, N, K = 300, 8192, 4096  # 10^10 elements, 5 GB of codes
    w = m.Mxfp4Weights(E, N, K, dev)
    w.codes.view(torch.int32).random_()
    w.scales.fill_(127)
    one = m.Mxfp4Weights(1, N, K, dev)
    one.codes.copy_(w.codes[-one.codes.numel():])
    one.scales.copy_(w.scales[-one.scales.numel():])
    for rows in (6, 300):
        x = torch.randn(rows, K, device=dev).to(torch.bfloat16)
        off = torch.zeros(E + 1, dtype=torch.int32, device=dev)
        off[E] = rows
        assert torch.equal(m.mxfp4_grouped_linear(x, off, w), m.mxfp4_linear(x, one))


def test_clip_past_32_bits(gpu):
    import torch
    m, dev = gpu
    n = (1 << 32) + 77
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device=dev)
    norm = float(m.clip_grad_norm(m.GradSet([g]), 1.0))
    assert abs(norm - 0.5 * n ** 0.5) <= 1e-12 * norm
    want = torch.tensor(0.5 / norm, dtype=torch.float64).float().to(torch.bfloat16)
    assert bool((g[-100:] == want.to(dev)).all()) and bool((g[:100] == want.to(dev)).all()) and float(g.min()) == float(g.max())


@pytest.mark.parametrize("T,E,k", [((1 << 28) + 21, 2, 1), ((1 << 26) + 7, 17, 17)])
def test_select_more_tokens_than_one_launch_takes(gpu, T, E, k):
    """16 lanes a token reach 2^32 work-items at 2^28 tokens, 64 lanes (17 slots) at 2^26."""
    import torch
    m, dev = gpu
    n = 1 << 20
    block = torch.randn(n, E, device=dev).to(torch.bfloat16)
    l = block.repeat(T // n, 1)
    l = torch.cat([l, block[:T - len(l)]])
    ids, probs = m.router_select(l, k)
    want, p = m.router_select(block, k)
    dp = torch.randn(n, k, device=dev)
    back = m.router_select_backward(block, want, dp, renormalize=False)
    dps = torch.cat([dp.repeat(T // n, 1), dp[:T - T // n * n]])
    got = m.router_select_backward(l, ids, dps, renormalize=False)
    for t in range(0, T, n):
        h = min(n, T - t)
        for a, b in ((ids, want), (probs, p), (got, back)):
            assert torch.equal(a[t:t + h], b[:h]), t
