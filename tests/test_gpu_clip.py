"""GPU gradient clipping (nvfp4moe_clip_grad_norm) against FP64.

Bars: the norm within 1e-13 relative (FP64 sums of n <= 10^7 squares in chains of at most some hundred additions); each
output bit for bit the FP64 product g * coef of the norm that was returned, rounded to FP32 and in BF16 tensors then to
BF16."""
import numpy as np
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


def _grads(sizes, dev, seed=0, scale=1e-2):
    """Contiguous tensors of these sizes, FP32 and BF16 in turn, at odd offsets of larger ones."""
    import torch
    g = torch.Generator(device=dev).manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = (torch.randn(n + 8, generator=g, device=dev) * scale).to(torch.bfloat16 if i % 2 else torch.float32)
        out.append(t[i % 5:i % 5 + n])
    return out


def _norm(grads):
    import torch
    return float(torch.stack([g.double().square().sum() for g in grads]).sum().sqrt())


def _scaled(g, norm, max_norm):
    coef = max_norm / norm if np.isfinite(norm) and norm > max_norm else 1.0
    return (g.double() * coef).float().to(g.dtype)


def _same(a, b):
    import torch
    return torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                       b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))


SIZES = [[1], [2, 3], [5, 7, 1, 8, 31, 33], [1023, 1025, 4099], [32768, 32769, 65537, 100003], [0, 5, 0, 300],
         [3 * 32768 + 5] * 3, list(range(1, 301)), [1 << 22, 999999]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("max_norm", [1e-3, 1e9])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip(gpu, sizes, max_norm, in_place):
    import torch
    m, dev = gpu
    grads = _grads(sizes, dev)
    before = [g.clone() for g in grads]
    out = None if in_place else [torch.full((g.numel() + 3,), 5.0, device=dev, dtype=g.dtype)[(i % 3):(i % 3) + g.numel()]
                                 for i, g in enumerate(grads)]
    norm = float(m.clip_grad_norm(m.GradSet(grads, out), max_norm))
    assert abs(norm - _norm(before)) <= 1e-13 * norm
    for i, (b, o) in enumerate(zip(before, grads if in_place else out)):
        assert _same(o, _scaled(b, norm, max_norm)), i
    if not in_place:
        assert all(_same(g, b) for g, b in zip(grads, before))


def test_neighbours_are_untouched(gpu):
    import torch
    m, dev = gpu
    for dtype in (torch.float32, torch.bfloat16):
        base = torch.full((5000,), 9.0, device=dev, dtype=dtype)
        parts = [base[3:1000], base[1001:1002], base[1003:4997]]
        norm = float(m.clip_grad_norm(m.GradSet(parts), 1.0))
        want = torch.full((5000,), 9.0, device=dev, dtype=dtype)
        for a, b in ((3, 1000), (1001, 1002), (1003, 4997)):
            want[a:b] = _scaled(want[a:b], norm, 1.0)
        assert torch.equal(base, want)


def test_extreme_values(gpu):
    """Squares that FP32 cannot hold, subnormals, a zero gradient, a limit of zero, the norm alone."""
    import torch
    m, dev = gpu
    big = torch.full((1000,), 3e38, device=dev)
    norm = float(m.clip_grad_norm(m.GradSet([big]), 1.0))
    assert abs(norm - 3e38 * np.sqrt(1000.0)) < 1e-6 * norm and torch.isfinite(big).all()
    tiny = torch.full((77,), 1e-44, device=dev)
    keep = tiny.clone()
    norm = float(m.clip_grad_norm(m.GradSet([tiny]), 1.0))
    assert abs(norm - float(keep[0].double()) * np.sqrt(77.0)) <= 1e-13 * norm and torch.equal(tiny, keep)
    zero = torch.zeros(50, device=dev)
    assert float(m.clip_grad_norm(m.GradSet([zero]), 0.0)) == 0.0 and (zero == 0).all()
    g = torch.randn(333, device=dev)
    keep = g.clone()
    norm = float(m.clip_grad_norm(m.GradSet([g]), float("inf")))
    assert abs(norm - _norm([keep])) <= 1e-13 * norm and torch.equal(g, keep)
    m.clip_grad_norm(m.GradSet([g]), 0.0)
    assert (g == 0).all()
    assert float(m.clip_grad_norm(m.GradSet([torch.empty(0, device=dev)]), 1.0)) == 0.0


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_nonfinite_gradients_are_left(gpu, bad):
    import torch
    m, dev = gpu
    grads = _grads([40000, 1001], dev)
    grads[1][500] = bad
    before = [g.clone() for g in grads]
    out = [torch.zeros(g.numel(), device=dev, dtype=g.dtype) for g in grads]
    norm = float(m.clip_grad_norm(m.GradSet(grads, out), 1e-3))
    assert not np.isfinite(norm)
    assert all(torch.equal(o.nan_to_num(5.0), b.nan_to_num(5.0)) for o, b in zip(out, before))
    m.clip_grad_norm(m.GradSet(grads), 1e-3)
    assert all(_same(g, b) for g, b in zip(grads, before))


def test_same_bits_every_run_stream_and_graph(gpu):
    import torch
    m, dev = gpu
    grads = _grads([100003, 7, 65536 * 3 + 1, 12], dev)
    out = [torch.empty_like(g) for g in grads]
    s = m.GradSet(grads, out)
    first = m.clip_grad_norm(s, 0.5)
    for _ in range(3):
        assert torch.equal(m.clip_grad_norm(s, 0.5), first)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream())
    again = m.clip_grad_norm(s, 0.5, stream=side)
    side.synchronize()
    assert torch.equal(again, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = m.clip_grad_norm(s, 0.5)
    for k in range(3):
        for g in grads:
            g.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        assert abs(float(norm) - _norm(grads)) <= 1e-13 * float(norm)
        assert all(_same(o, _scaled(g, float(norm), 0.5)) for g, o in zip(grads, out))


def test_refusals(gpu):
    import torch
    m, dev = gpu
    g = torch.zeros(100, device=dev)
    for grads, out in (([g, g], None), ([g[:60], g[50:]], None), ([g[:50]], [g[10:60]])):
        with pytest.raises(m.Nvfp4Error):
            m.GradSet(grads, out)
    with pytest.raises(ValueError):
        m.GradSet([g], [g.to(torch.bfloat16)])
    with pytest.raises(m.Nvfp4Error):
        m.clip_grad_norm(m.GradSet([g]), -1.0)


@pytest.mark.parametrize("max_norm", [1e-3, float("inf")])
def test_nonfinite_gradients_are_copied_to_the_bit(gpu, max_norm):
    """Outputs apart from the inputs, aligned with them and not: signaling and quiet NaNs keep every bit."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(17)
    for kind, bits, nans in ((torch.float32, torch.int32, (0x7F800001, -0x7FFFFF, 0x7FC12345, -1, 0x7F800000)),
                             (torch.bfloat16, torch.int16, (0x7F81, -0x7F, 0x7FD5, -1, 0x7F80))):
        for shift in (0, 1):
            g = torch.randn(5000, device=dev).to(kind)[3:]
            at = torch.from_numpy(rng.choice(4997, 400, replace=False)).to(dev)
            g.view(bits)[at] = torch.tensor(nans, dtype=bits, device=dev).repeat(80)
            g.view(bits)[0] = nans[0]
            out = torch.zeros(5001, device=dev, dtype=kind)[3 + shift:][:4997]
            assert not np.isfinite(float(m.clip_grad_norm(m.GradSet([g], [out]), max_norm)))
            assert torch.equal(out.view(bits), g.view(bits))
