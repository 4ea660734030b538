"""GPU low-rank adapters (nvfp4moe_adapter_linear) and their gradients against FP64.

Whole numbers: every product and sum is exact in FP32, v in two BF16 values, so the outputs are the exact ones rounded
once, to the bit.  Other values: the bounds derived in plain_train_ops.adapter_linear and adapter_backward, and one
rounding of the output's type."""
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


def _whole(M, K, N, rank, n, dev, seed=0, most=2):
    """Whole numbers of at most `most`; the scales are powers of two."""
    import torch
    g = torch.Generator(device=dev).manual_seed(seed)

    def ints(*shape, top=most):
        return torch.randint(-top, top + 1, shape, generator=g, device=dev).to(torch.bfloat16)

    ids = torch.randint(-1, n, (M,), generator=g, device=dev).to(torch.int32)
    return dict(x=ints(M, K), ids=ids, A=ints(n, rank, K, top=1), B=ints(n, N, rank, top=1),
                scale=2.0 ** torch.randint(-1, 2, (n,), generator=g, device=dev).float(), base=ints(M, N, top=100)), g


def _bf16(t):
    """FP64 values that FP32 holds, rounded to BF16."""
    import torch
    assert torch.equal(t.float().double(), t)
    return t.float().to(torch.bfloat16)


SIZES = [(1, 8, 8, 8, 1), (1, 2048, 4096, 16, 8), (5, 72, 40, 8, 3), (7, 512, 264, 24, 2), (16, 64, 64, 16, 1),
         (17, 1000, 1544, 32, 4), (33, 136, 528, 40, 3), (64, 4096, 512, 64, 5), (100, 520, 72, 72, 7), (130, 256, 1032, 128, 2),
         (200, 96, 4104, 16, 64), (256, 640, 640, 32, 300), (257, 640, 640, 16, 3), (1000, 264, 200, 96, 9),
         (3001, 128, 192, 16, 1024), (2500, 512, 1024, 64, 2), (5000, 72, 88, 8, 1)]


@pytest.mark.parametrize("M,K,N,rank,n", SIZES)
def test_whole_numbers(gpu, M, K, N, rank, n):
    import torch
    m, dev = gpu
    t, _ = _whole(M, K, N, rank, n, dev, M + K)
    v = torch.full((M, rank), 9.0, device=dev)
    got = m.adapter_linear(**t, v=v)
    out, want_v, _ = R.adapter_linear(**t)
    assert torch.equal(got, _bf16(out))
    assert torch.equal(v.double(), want_v)
    t["base"] = None
    assert torch.equal(m.adapter_linear(**t), _bf16(R.adapter_linear(**t)[0]))
    t["scale"] = None
    assert torch.equal(m.adapter_linear(**t), _bf16(R.adapter_linear(**t)[0]))


@pytest.mark.parametrize("M,K,N,rank,n", SIZES)
def test_whole_number_gradients(gpu, M, K, N, rank, n):
    import torch
    m, dev = gpu
    t, g = _whole(M, K, N, rank, n, dev, M + N)
    base = torch.randint(-100, 101, (M, K), generator=g, device=dev).to(torch.bfloat16)
    dy = torch.randint(-2, 3, (M, N), generator=g, device=dev).to(torch.bfloat16)
    v = torch.randint(-2000, 2001, (M, rank), generator=g, device=dev).float()
    for b, scale in ((base, t["scale"]), (None, None)):
        args = (t["x"], t["ids"], t["A"], t["B"], v, dy, b, scale)
        got = m.adapter_backward(*args)
        want, _ = R.adapter_backward(*args)
        assert float(want[1].abs().max()) < 2 ** 24 and float(want[2].abs().max()) < 2 ** 24
        assert torch.equal(got[0], _bf16(want[0]))
        assert torch.equal(got[1].double(), want[1]) and torch.equal(got[2].double(), want[2])


def _float(M, K, N, rank, n, dev, seed=0):
    import torch
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(torch.bfloat16)

    ids = torch.randint(-1, n, (M,), generator=g, device=dev).to(torch.int32)
    return dict(x=randn(M, K), ids=ids, A=randn(n, rank, K, std=K ** -0.5), B=randn(n, N, rank, std=0.1),
                scale=torch.rand(n, generator=g, device=dev) * 3 - 1, base=randn(M, N)), g, randn


@pytest.mark.parametrize("M,K,N,rank,n", [(3, 2048, 4096, 16, 2), (61, 4096, 520, 64, 3), (500, 1032, 264, 128, 4),
                                          (2000, 520, 1544, 24, 3)])
def test_real_numbers(gpu, M, K, N, rank, n):
    import torch
    m, dev = gpu
    t, g, randn = _float(M, K, N, rank, n, dev, M)
    v = torch.empty(M, rank, device=dev)
    got = m.adapter_linear(**t, v=v)
    out, want_v, bound = R.adapter_linear(**t)
    assert ((got.double() - out).abs() <= bound * (1 + R.BF16) + R.BF16 * out.abs()).all()
    a = t["ids"].long().clamp(min=0)
    mag = torch.stack([t["x"][r].double().abs() @ t["A"][a[r]].double().abs().t() for r in range(M)])
    assert ((v.double() - want_v).abs() <= R.chain(K / 256) * mag).all()
    dy, base = randn(M, N), randn(M, K)
    args = (t["x"], t["ids"], t["A"], t["B"], v, dy, base, t["scale"])
    got, (want, bounds) = m.adapter_backward(*args), R.adapter_backward(*args)
    assert ((got[0].double() - want[0]).abs() <= bounds[0] * (1 + R.BF16) + R.BF16 * want[0].abs()).all()
    for k in (1, 2):
        assert ((got[k].double() - want[k]).abs() <= bounds[k] + R.U * want[k].abs()).all()


def test_gradient_against_differences(gpu):
    """The forward pass is linear in each of x, A and B: with whole numbers, differences are exact."""
    import torch
    m, dev = gpu
    M, K, N, rank, n = 37, 64, 72, 16, 3
    t, g = _whole(M, K, N, rank, n, dev, 1, most=1)
    t["base"] = None
    dy = torch.randint(-1, 2, (M, N), generator=g, device=dev).to(torch.bfloat16)
    v = torch.empty(M, rank, device=dev)
    m.adapter_linear(**t, v=v)
    dx, dA, dB = m.adapter_backward(t["x"], t["ids"], t["A"], t["B"], v, dy, scale=t["scale"])
    for name, grad in (("x", dx), ("A", dA), ("B", dB)):
        e = torch.randint(-1, 2, t[name].shape, generator=g, device=dev).to(torch.bfloat16)
        up, down = (R.adapter_linear(**(t | {name: t[name] + s * e}))[0] for s in (1, -1))
        slope = float(((up - down) / 2 * dy.double()).sum())
        assert slope == float((grad.double() * e.double()).sum())


def test_rows_do_not_depend_on_the_batch(gpu):
    """Each row's bits alone, in batches that take every path, at another place, and beside rows of NaN."""
    import torch
    m, dev = gpu
    for rank in (8, 16, 32, 64, 128):
        t, g, _ = _float(700, 1544, 584, rank, 3, dev, rank)
        v = torch.empty(700, rank, device=dev)
        whole = m.adapter_linear(**t, v=v)
        for rows in ([0], [699], list(range(5)), list(range(100, 117)), list(range(0, 250)), list(range(0, 600, 2)),
                     list(range(699, -1, -1))):
            i = torch.tensor(rows, device=dev)
            part = {k: t[k][i].contiguous() if k in ("x", "ids", "base") else t[k] for k in t}
            vp = torch.empty(len(rows), rank, device=dev)
            assert torch.equal(m.adapter_linear(**part, v=vp), whole[i]) and torch.equal(vp, v[i])
        bad = torch.zeros(700, dtype=torch.bool, device=dev)
        bad[::7] = True
        t["x"][bad] = float("nan")
        got = m.adapter_linear(**t)
        assert torch.equal(got[~bad], whole[~bad])
        live = bad & (t["ids"] >= 0)
        assert torch.isnan(got[live]).all() and torch.equal(got[bad & ~live], whole[bad & ~live])


@pytest.mark.parametrize("M", [9, 300])
def test_rows_without_an_adapter(gpu, M):
    """Ids outside the adapters: base to the bit (NaN and -0 among it), whatever x holds."""
    import torch
    m, dev = gpu
    t, _ = _whole(M, 64, 72, 16, 4, dev, 2)
    t["ids"][:5] = torch.tensor([-1, 4, 2 ** 31 - 1, -2 ** 31, 1000], device=dev)
    t["x"][:5] = float("inf")
    t["base"][0] = -0.0
    t["base"].view(torch.int16)[1] = 0x7F81
    v = torch.full((M, 16), 5.0, device=dev)
    got = m.adapter_linear(**t, v=v)
    assert torch.equal(got[:5].view(torch.int16), t["base"][:5].view(torch.int16)) and not v[:5].any()
    none = dict(t, ids=torch.full_like(t["ids"], -1))
    assert torch.equal(m.adapter_linear(**none).view(torch.int16), t["base"].view(torch.int16))
    keep = t["base"].clone()
    assert m.adapter_linear(**dict(none, base=keep), out=keep) is keep
    assert torch.equal(keep.view(torch.int16), t["base"].view(torch.int16))
    assert not m.adapter_linear(**dict(none, base=None)).any()
    dy = torch.ones(M, 72, dtype=torch.bfloat16, device=dev)
    dxb = torch.randn(M, 64, device=dev).to(torch.bfloat16)
    dx, dA, dB = m.adapter_backward(none["x"], none["ids"], t["A"], t["B"], v, dy, dxb, t["scale"])
    assert torch.equal(dx, dxb) and not dA.any() and not dB.any()


def test_infinite_rows_and_low_ranks(gpu):
    """An infinite x gives what the definition gives, also where the rank is padded inside the kernel."""
    import torch
    m, dev = gpu
    for M in (3, 300):
        x = torch.ones(M, 64, dtype=torch.bfloat16, device=dev)
        x[1, 5] = float("inf")
        A = torch.ones(1, 8, 64, dtype=torch.bfloat16, device=dev)
        B = torch.ones(1, 40, 8, dtype=torch.bfloat16, device=dev)
        ids = torch.zeros(M, dtype=torch.int32, device=dev)
        out = m.adapter_linear(x, ids, A, B)
        assert (out[1] == float("inf")).all() and (out[0] == 512).all() and (out[2:] == 512).all()


def test_strides_in_place_and_neighbours(gpu):
    import torch
    m, dev = gpu
    for M in (40, 500):
        t, g = _whole(M, 136, 200, 24, 5, dev, M)
        want = m.adapter_linear(**t)
        big_x = torch.full((M, 160), float("nan"), dtype=torch.bfloat16, device=dev)
        big_x[:, 8:144] = t["x"]
        big = torch.full((M + 2, 224), 7.0, dtype=torch.bfloat16, device=dev)
        view = big[1:M + 1, 16:216]
        view.copy_(t["base"])
        args = dict(t, x=big_x[:, 8:144], base=view)
        assert m.adapter_linear(**args, out=view) is view
        assert torch.equal(view, want)
        view.fill_(7.0)
        assert (big == 7).all()
        dy = torch.randint(-2, 3, (M, 200), generator=g, device=dev).to(torch.bfloat16)
        v = torch.randint(-9, 10, (M, 24), generator=g, device=dev).float()
        dxb = torch.randint(-9, 10, (M, 136), generator=g, device=dev).to(torch.bfloat16)
        ref = m.adapter_backward(t["x"], t["ids"], t["A"], t["B"], v, dy, dxb, t["scale"])
        big_dy = torch.full((M, 208), float("nan"), dtype=torch.bfloat16, device=dev)
        big_dy[:, :200] = dy
        big_dx = torch.full((M, 144), 7.0, dtype=torch.bfloat16, device=dev)
        big_dx[:, :136] = dxb
        out = (big_dx[:, :136], torch.full_like(ref[1], 3.0), torch.full_like(ref[2], 3.0))
        got = m.adapter_backward(big_x[:, 8:144], t["ids"], t["A"], t["B"], v, big_dy[:, :200], big_dx[:, :136], t["scale"], out)
        assert all(torch.equal(a, b) for a, b in zip(got, ref)) and (big_dx[:, 136:] == 7).all()


@pytest.mark.parametrize("M", [3, 200, 3000])
def test_same_bits_every_run_stream_and_graph(gpu, M):
    import torch
    m, dev = gpu
    t, g, randn = _float(M, 264, 520, 16, 3, dev, M)
    dy, dxb = randn(M, 520), randn(M, 264)
    v = torch.empty(M, 16, device=dev)
    ws = m.adapter_alloc_workspace(M, 264, 520, 16, 3, backward=True, device=dev)

    def step(stream=None):
        out = m.adapter_linear(**t, v=v, workspace=ws, stream=stream)
        return (out, *m.adapter_backward(t["x"], t["ids"], t["A"], t["B"], v, dy, dxb, t["scale"], workspace=ws, stream=stream))

    first = step()
    side = torch.cuda.Stream(dev)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, step()))
        side.wait_stream(torch.cuda.current_stream())
        again = step(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        t["x"].mul_(-1.25)
        t["ids"].copy_(torch.randint(-1, 3, (M,), generator=g, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        mine = [x.clone() for x in got]
        assert all(torch.equal(a, b) for a, b in zip(mine, step()))


def test_no_rows(gpu):
    import torch
    m, dev = gpu
    t, _ = _whole(0, 64, 72, 16, 4, dev)
    assert m.adapter_linear(**t).shape == (0, 72)
    dx, dA, dB = m.adapter_backward(t["x"], t["ids"], t["A"], t["B"], torch.empty(0, 16, device=dev), t["base"])
    assert dx.shape == (0, 64) and not dA.any() and not dB.any()


def test_refusals(gpu):
    import torch
    m, dev = gpu
    t, _ = _whole(6, 64, 72, 16, 4, dev)

    def bad(error, **kw):
        with pytest.raises(error):
            m.adapter_linear(**(t | kw))

    bad(ValueError, ids=t["ids"].long())
    bad(ValueError, ids=t["ids"][:5])
    bad(ValueError, x=t["x"].float())
    bad(ValueError, A=t["A"][:, :, ::2])
    bad(ValueError, B=t["B"].transpose(1, 2))
    bad(ValueError, base=t["base"][:, :64])
    bad(ValueError, scale=t["scale"].double())
    bad(ValueError, v=torch.empty(6, 15, device=dev))
    bad(m.Nvfp4Error, workspace=torch.empty(256, dtype=torch.uint8, device=dev))
    bad(m.Nvfp4Error, x=torch.zeros(6, 68, dtype=torch.bfloat16, device=dev)[:, 4:])  # not 16-byte aligned
    bad(m.Nvfp4Error, A=t["A"][:, :12].contiguous(), B=t["B"][:, :, :12].contiguous())  # rank 12
    with pytest.raises(ValueError):
        m.adapter_linear(**{k: x.cpu() for k, x in t.items()})
    with pytest.raises(m.Nvfp4Error):
        m.adapter_alloc_workspace(5, 64, 72, 136, 1)
    with pytest.raises(ValueError):
        m.adapter_backward(t["x"], t["ids"], t["A"], t["B"], torch.empty(6, 16, device=dev), t["x"])
