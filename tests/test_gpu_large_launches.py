"""Calls of so many rows that one launch would have 2^32 threads or more along an axis, of which HIP runs none and
reports no error."""
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


def _repeated(t, rows):
    """The rows of t again and again."""
    import torch
    out = torch.empty(rows, *t.shape[1:], dtype=t.dtype, device=t.device)
    for r in range(0, rows, t.shape[0]):
        out[r:r + t.shape[0]] = t[:rows - r]
    return out


@pytest.mark.parametrize("layout", ["logical", "gemm"])
def test_quantizer(gpu, layout):
    """A wavefront a row of 16 columns; eight rows of 128 a wavefront, in row tiles of 32 (more than one launch takes)."""
    import torch
    m, dev = gpu
    P, cols, which = 1 << 20, *((16, m.LAYOUT_LOGICAL) if layout == "logical" else (128, m.LAYOUT_GEMM))
    rows = (1 << 26) + (3 if layout == "logical" else 32)
    few = (torch.randn(P, cols, device=dev) * 2.0 ** torch.randint(-8, 9, (P, 1), device=dev)).to(torch.bfloat16)
    x = _repeated(few, rows)
    want, got = m.quantize(few, which), m.quantize(x, which)
    for a, b in zip(got, want):
        a, b = a.view(-1), b.view(-1)
        each, times, rest = b.numel(), rows // P, rows % P
        assert a.numel() == times * each + rest * (each // P)
        assert (a[:times * each].view(times, each) == b).all() and torch.equal(a[times * each:], b[:rest * (each // P)])


def test_router_topk(gpu):
    """A wavefront a token."""
    import torch
    m, dev = gpu
    P, T, H, E, k = 1 << 20, (1 << 26) + 5, 16, 4, 2
    few, w = torch.randn(P, H, device=dev).to(torch.bfloat16), torch.randn(E, H, device=dev).to(torch.bfloat16)
    want, got = m.router_topk(few, w, k), m.router_topk(_repeated(few, T), w, k)
    for a, b in zip(got, want):
        assert torch.equal(a, _repeated(b, T))
