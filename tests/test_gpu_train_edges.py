"""The balance loss and the low-rank adapters where a value, a size or a list of sequences is out of the ordinary."""
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


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 96, 128])
@pytest.mark.parametrize("M", [3, 600, 5000])
def test_all_bits_of_v_reach_the_outputs(gpu, M, rank):
    """v = 1 + 2^-12 + 2^-22 in one rank, -2^-12 in another and a base of -1: out is 2^-22.  Every sum on the way fits
    FP32, in whatever order; a v of 16 bits would give 0.  The gradient's dx likewise."""
    import torch
    m, dev = gpu
    K, N = 136, 200

    def small(wide):  # one row of inputs, and the two adapter rows that make v of it
        z = torch.zeros(rank, wide)
        z[rank - 1, :3] = torch.tensor([1.0, 1.0, 1.0])
        z[0, wide - 1] = -1.0
        x = torch.zeros(wide)
        x[:3], x[wide - 1] = torch.tensor([1.0, 2.0 ** -12, 2.0 ** -22]), 2.0 ** -12
        return x, z

    ids = torch.arange(M, dtype=torch.int32, device=dev) % 2
    (x, a), (dy, b) = small(K), small(N)
    x, dy = (t.to(torch.bfloat16).to(dev).expand(M, -1).contiguous() for t in (x, dy))
    ones = torch.zeros(rank)
    ones[0] = ones[rank - 1] = 1.0
    A = a.expand(2, -1, -1).to(torch.bfloat16).to(dev).contiguous()
    B = ones.expand(2, N, -1).to(torch.bfloat16).to(dev).contiguous()
    base = torch.full((M, N), -1.0, dtype=torch.bfloat16, device=dev)
    v = torch.empty(M, rank, device=dev)
    out = m.adapter_linear(x, ids, A, B, base, v=v)
    assert (v[:, rank - 1] == 1 + 2.0 ** -12 + 2.0 ** -22).all() and (v[:, 0] == -2.0 ** -12).all()
    assert (out == 2.0 ** -22).all(), out.unique()
    # dx = base + A^T B^T dy, A of ones in the same two ranks
    A = ones[:, None].expand(2, -1, K).to(torch.bfloat16).to(dev).contiguous()
    B = b.t().expand(2, -1, -1).to(torch.bfloat16).to(dev).contiguous()
    dx = m.adapter_backward(x, ids, A, B, v, dy, torch.full((M, K), -1.0, dtype=torch.bfloat16, device=dev))[0]
    assert (dx == 2.0 ** -22).all(), dx.unique()
