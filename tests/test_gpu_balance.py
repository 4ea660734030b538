"""GPU balance loss (nvfp4moe_router_balance_loss) and its gradient against FP64.

Bars, with u = 2^-24: counts equal; the loss is a sum of positive terms, each probability within 12 u by its
exponential and reciprocal and 12 u by the token's sum's, then FP32 sums of at most 22 (a token's lane), 6 (its lanes),
16 (tokens of a lane) and 16 (lanes) terms: 96 u relative and one rounding; the gradient's bound is derived in
plain_train_ops.balance_backward, with half a step of the output's type."""
import pytest

from tests import plain_train_ops as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_moe_expert_sort_amd as m
    m.lib()
    return m, torch.device("cuda:0")


def _inputs(T, E, k, dev, seed=0, bf16=False, spread=1.5):
    import torch
    g = torch.Generator(device=dev).manual_seed(seed)
    l = (torch.randn(T, E, generator=g, device=dev) * spread + torch.randn(1, E, generator=g, device=dev)).to(
        torch.bfloat16 if bf16 else torch.float32)
    ids = torch.randint(0, E, (T, k), generator=g, device=dev).to(torch.int32)
    return l, ids, g


def _offsets(T, S, g, dev):
    import torch
    cut = (torch.rand(S - 1, generator=g, device=dev) * (T + 1)).long().clamp(max=T).sort()[0].int()
    ends = torch.tensor([0, T], dtype=torch.int32, device=dev)
    return torch.cat([ends[:1], cut, ends[1:]])


def _check(m, l, ids, offsets, sigmoid, coef=0.01, add=None, dloss=None):
    import torch
    score = m.SCORE_SIGMOID if sigmoid else m.SCORE_SOFTMAX
    loss, counts = m.router_balance_loss(l, ids, coef, score=score, offsets=offsets)
    want, n = R.balance_loss(l, ids, coef, sigmoid, offsets)
    assert torch.equal(counts.long(), n)
    assert abs(float(loss) - want) <= 97 * R.U * abs(want), (float(loss), want)
    got = m.router_balance_backward(l, counts, ids.shape[1], coef, score=score, offsets=offsets, add=add, dloss=dloss)
    d, bound = R.balance_backward(l, counts, ids.shape[1], coef, sigmoid, offsets,
                                  1.0 if dloss is None else float(dloss), add)
    last = (R.BF16 + 2 * R.U if l.dtype == torch.bfloat16 else 2 * R.U) * (d.abs() + bound)
    err = (got.double() - d).abs()
    assert (err <= bound + last + 1e-40).all(), float((err / (bound + last + 1e-40)).max())
    return loss, counts, got


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (3, 5, 2), (16, 64, 4), (17, 65, 1), (61, 128, 8), (300, 129, 3),
                                   (1000, 250, 7), (4099, 256, 8), (37, 257, 32), (515, 512, 10), (130, 1000, 8),
                                   (70, 1024, 2)])
def test_sizes(gpu, T, E, k, sigmoid):
    import torch
    m, dev = gpu
    for bf16 in (False, True):
        l, ids, g = _inputs(T, E, k, dev, T + E, bf16)
        add = torch.randn(T, E, generator=g, device=dev).mul(1e-5).to(l.dtype)
        _check(m, l, ids, None, sigmoid, add=add, dloss=torch.full((1,), 0.37, device=dev))


@pytest.mark.parametrize("T,E,S", [(1, 8, 3), (40, 16, 40), (50, 128, 7), (50, 33, 200), (3000, 256, 13), (5000, 100, 64),
                                   (777, 600, 5)])
def test_sequences(gpu, T, E, S):
    m, dev = gpu
    for sigmoid in (False, True):
        l, ids, g = _inputs(T, E, 4, dev, S)
        off = _offsets(T, S, g, dev)
        _, counts, _ = _check(m, l, ids, off, sigmoid)
        assert int(counts.sum()) == 4 * T


def test_rows_outside_the_sequences(gpu):
    """Rows before the first offset and from the last one on, sequences without rows, offsets out of range."""
    import torch
    m, dev = gpu
    l, ids, _ = _inputs(100, 24, 3, dev, 5)
    add = torch.randn(100, 24, device=dev)
    for off in ([7, 7, 30, 30, 64, 91], [0, 0], [100, 100, 100], [50, 50], [-5, 20, 500], [99, 100], [0, 1]):
        o = torch.tensor(off, dtype=torch.int32, device=dev)
        _, _, d = _check(m, l, ids, o, False)
        _, _, e = _check(m, l, ids, o, True, add=add)
        a, b = min(max(off[0], 0), 100), min(off[-1], 100)
        assert not d[:a].any() and not d[b:].any()
        assert torch.equal(e[:a], add[:a]) and torch.equal(e[b:], add[b:])


def test_unusable_logits_and_ids(gpu):
    """NaN, infinities, the type's lowest value, rows masked whole, ids outside the experts."""
    import torch
    m, dev = gpu
    T, E = 64, 40
    inf = float("inf")
    for kind in (torch.float32, torch.bfloat16):
        l, ids, _ = _inputs(T, E, 4, dev, 9, kind == torch.bfloat16)
        low = torch.finfo(kind).min
        l[0] = -inf
        l[1] = float("nan")
        l[2] = low
        l[3, ::2] = -inf
        l[4, 1::3] = low
        l[5, 7] = inf
        l[6, 3:] = float("nan")
        l[7, 1:] = -inf
        l[8] = -1e4
        l[9] = 1e4
        l[10] = -torch.arange(E, device=dev).to(kind) * 200
        l[11] = -3e38
        l[12, 0] = 3e38
        ids[13] = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31], device=dev)
        ids[14] = 5
        for sigmoid in (False, True):
            _, _, d = _check(m, l, ids, None, sigmoid)
            assert torch.isfinite(d).all()
            assert not d[0].any() and not d[1].any() and not d[3, ::2].any() and not d[6, 3:].any()


def test_confident_tokens(gpu):
    """One expert with nearly all the probability: the gradient is a small difference that must not be lost."""
    import torch
    m, dev = gpu
    l, ids, _ = _inputs(200, 64, 4, dev, 11, spread=0.1)
    l[torch.arange(200), torch.randint(0, 64, (200,), device=dev)] += torch.linspace(5, 60, 200, device=dev)
    for sigmoid in (False, True):
        _check(m, l, ids, None, sigmoid)


def test_gradient_against_differences(gpu):
    """(loss(l + h e) - loss(l - h e)) / 2h of the kernel's FP32 loss, along the gradient.  The loss is within 97 u of its
    value.  Along a direction of norm r in a token's logits, with c = e - mean e (|c| <= sqrt(2) r), the third derivative
    of p is p (c^3 - 3 c var - third moment), in sum at most 5 (sqrt(2) r)^3 = 14 r^3; a sigmoid's own curvature, whose
    logarithm's derivatives are at most 1, 1/4 and 1/8 of those, keeps it below 40 r^3.  h^2 / 6 of it remains."""
    import torch
    m, dev = gpu
    l, ids, g = _inputs(33, 16, 2, dev, 3)
    off = torch.tensor([0, 9, 20, 33], dtype=torch.int32, device=dev)
    ids[:] = torch.randint(0, 3, ids.shape, generator=g, device=dev)  # an uneven load
    h = 2.0 ** -6
    for score in (m.SCORE_SOFTMAX, m.SCORE_SIGMOID):
        loss, counts = m.router_balance_loss(l, ids, 1.0, score=score, offsets=off)
        d = m.router_balance_backward(l, counts, 2, 1.0, score=score, offsets=off)
        e = d / d.norm()
        up, down = (float(m.router_balance_loss(l + s * h * e, ids, 1.0, score=score, offsets=off)[0]) for s in (1, -1))
        slope, want = (up - down) / (2 * h), float((d * e).sum())
        f = float((counts.double() * 16 / 2 / (off[1:] - off[:-1])[:, None]).max())
        bar = 2 * 97 * R.U * float(loss) / (2 * h) + 7 * h * h * f * float((e.norm(dim=1) ** 3).sum()) / 33
        assert abs(slope - want) <= bar and want > 10 * bar, (slope, want, bar)


@pytest.mark.parametrize("bf16", [False, True])
def test_strides_and_in_place(gpu, bf16):
    import torch
    m, dev = gpu
    kind = torch.bfloat16 if bf16 else torch.float32
    for E, wide in ((20, 33), (128, 200), (256, 260), (600, 601)):
        l, ids, g = _inputs(77, E, 4, dev, E, bf16)
        big = torch.full((77, wide), 7.0, device=dev, dtype=kind)
        big[:, 1:1 + E] = l
        loss, counts = m.router_balance_loss(l, ids, 0.01)
        loss2, counts2 = m.router_balance_loss(big[:, 1:1 + E], ids, 0.01)
        assert torch.equal(loss, loss2) and torch.equal(counts, counts2)
        add = torch.randn(77, E, generator=g, device=dev).mul(1e-4).to(kind)
        want = m.router_balance_backward(l, counts, 4, 0.01, add=add)
        out = torch.full((77, wide), 3.0, device=dev, dtype=kind)
        out[:, 1:1 + E] = add
        view = out[:, 1:1 + E]
        assert m.router_balance_backward(big[:, 1:1 + E], counts, 4, 0.01, add=view, out=view) is view
        assert torch.equal(view, want)
        assert (out[:, 0] == 3).all() and (out[:, 1 + E:] == 3).all()


def test_same_bits_every_run_stream_and_graph(gpu):
    import torch
    m, dev = gpu
    l, ids, g = _inputs(3001, 128, 8, dev, 21)
    off = _offsets(3001, 9, g, dev)
    a = m.router_balance_loss(l, ids, 0.01, offsets=off)
    side = torch.cuda.Stream(dev)
    for _ in range(3):
        b = m.router_balance_loss(l, ids, 0.01, offsets=off)
        side.wait_stream(torch.cuda.current_stream())
        c = m.router_balance_loss(l, ids, 0.01, offsets=off, stream=side)
        side.synchronize()
        assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, counts = m.router_balance_loss(l, ids, 0.01, offsets=off)
        d = m.router_balance_backward(l, counts, 8, 0.01, offsets=off, dloss=loss)
    for _ in range(4):
        l.mul_(1.1)
        ids.copy_(torch.randint(0, 128, ids.shape, generator=g, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        want, n = m.router_balance_loss(l, ids, 0.01, offsets=off)
        assert torch.equal(loss, want) and torch.equal(counts, n)
        assert torch.equal(d, m.router_balance_backward(l, n, 8, 0.01, offsets=off, dloss=want))


def test_no_rows(gpu):
    import torch
    m, dev = gpu
    l, ids = torch.empty(0, 16, device=dev), torch.empty(0, 4, dtype=torch.int32, device=dev)
    for off in (None, torch.zeros(4, dtype=torch.int32, device=dev)):
        loss, counts = m.router_balance_loss(l, ids, 0.01, offsets=off)
        assert float(loss) == 0.0 and not counts.any() and counts.shape == (1 if off is None else 3, 16)
        assert m.router_balance_backward(l, counts, 4, 0.01, offsets=off).shape == (0, 16)


def test_refusals(gpu):
    import torch
    m, dev = gpu
    l, ids, _ = _inputs(8, 16, 2, dev)
    counts = torch.zeros(1, 16, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        m.router_balance_loss(l, ids.long(), 0.01)
    with pytest.raises(ValueError):
        m.router_balance_loss(l, ids[:7], 0.01)
    with pytest.raises(ValueError):
        m.router_balance_loss(l, ids, 0.01, offsets=torch.zeros(1, dtype=torch.int32, device=dev))
    with pytest.raises(ValueError):
        m.router_balance_loss(l.half(), ids, 0.01)
    with pytest.raises(ValueError):
        m.router_balance_loss(l.cpu(), ids.cpu(), 0.01)
    with pytest.raises(m.Nvfp4Error):
        m.router_balance_loss(l, ids, float("nan"))
    with pytest.raises(m.Nvfp4Error):
        m.router_balance_loss(l, ids, 0.01, score=2)
    with pytest.raises(ValueError):
        m.router_balance_backward(l, counts, 2, 0.01, add=l.to(torch.bfloat16))
    with pytest.raises(ValueError):
        m.router_balance_backward(l, counts, 2, 0.01, offsets=torch.zeros(3, dtype=torch.int32, device=dev))
    with pytest.raises(m.Nvfp4Error):  # in place, but with another stride
        buf = torch.zeros(300, device=dev)
        m.router_balance_backward(l, counts, 2, 0.01, add=buf[:8 * 16].view(8, 16), out=buf[:8 * 20].view(8, 20)[:, :16])
