"""The balance loss and the low-rank adapters in the runs they are made for (a fine-tuning step over quantized weights,
experts with adapters, both captured in a graph), at the sizes where their kernels change, past 32 bits, with the
workspace's and the outputs' neighbours watched, and on streams that are not the tensors' own."""
import copy

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


def _randn(g, *shape, std=1.0):
    import torch
    return (torch.randn(shape, generator=g, device=g.device) * std).to(torch.bfloat16)


def _near(got, want, bound):
    """One BF16 rounding behind the bound."""
    assert ((got.double() - want).abs() <= bound * (1 + R.BF16) + R.BF16 * want.abs()).all()


def _gradients_near(got, args):
    want, bounds = R.adapter_backward(*args)
    _near(got[0], want[0], bounds[0])
    for k in (1, 2):
        assert ((got[k].double() - want[k]).abs() <= bounds[k] + R.U * want[k].abs()).all()


def _balance_near(m, loss, counts, d, l, ids, coef, off, add):
    want, n = R.balance_loss(l, ids, coef, False, off)
    assert abs(float(loss) - want) <= 97 * R.U * want
    assert counts.tolist() == n.tolist()
    ref, bound = R.balance_backward(l, counts, ids.shape[1], coef, False, off, 1.0, add)
    assert ((d.double() - ref).abs() <= bound + 2 * R.U * (ref.abs() + bound) + 1e-40).all()


class _Step:
    """A fine-tuning step of a layer whose weights stay in MXFP4: router, selection and balance loss over packed
    sequences; a projection shared by all rows, with an adapter per request; gradients of router and adapters, clipped."""

    def __init__(self, m, dev, T, H, N, E, k, rank, n, seed):
        import torch
        g = torch.Generator(device=dev).manual_seed(seed)
        self.m, self.k, self.g = m, k, g
        self.x, self.wr, w = _randn(g, T, H), _randn(g, E, H, std=0.1), _randn(g, 1, N, H, std=H ** -0.5)
        self.W = m.Mxfp4Weights(1, N, H, dev).quantize_from(w)
        self.Wt = m.Mxfp4Weights(1, H, N, dev).quantize_from(w.transpose(1, 2).contiguous())
        self.A, self.B = _randn(g, n, rank, H, std=H ** -0.5), _randn(g, n, N, rank, std=0.1)
        self.scale = torch.rand(n, generator=g, device=dev) + 0.5
        self.dy, self.dprobs = _randn(g, T, N), torch.randn(T, k, generator=g, device=dev)
        self.off = torch.tensor([0, T // 3, T // 3, T - T // 8], dtype=torch.int32, device=dev)
        # a request's rows follow each other, the last ones have no adapter
        self.who = (torch.arange(T, device=dev) * (n + 1) // T).int()
        self.ws = m.adapter_alloc_workspace(T, H, N, rank, n, backward=True, device=dev)

    def forward(self):
        m = self.m
        self.l = m.router_logits(self.x, self.wr)
        self.ids, self.probs = m.router_select(self.l, self.k)
        self.loss, self.counts = m.router_balance_loss(self.l, self.ids, 0.01, offsets=self.off)
        self.y0 = m.mxfp4_linear(self.x, self.W)
        self.v = self.x.new_empty(self.x.shape[0], self.A.shape[1], dtype=self.scale.dtype)
        self.y = m.adapter_linear(self.x, self.who, self.A, self.B, self.y0, self.scale, v=self.v, workspace=self.ws)

    def backward(self):
        m = self.m
        self.dl0 = m.router_select_backward(self.l, self.ids, self.dprobs)
        self.dl = m.router_balance_backward(self.l, self.counts, self.k, 0.01, offsets=self.off, add=self.dl0)
        self.dx0 = m.mxfp4_linear(self.dy, self.Wt)
        self.grads = m.adapter_backward(self.x, self.who, self.A, self.B, self.v, self.dy, self.dx0, self.scale,
                                        workspace=self.ws)

    def check(self):
        import torch
        _balance_near(self.m, self.loss, self.counts, self.dl, self.l, self.ids, 0.01, self.off, self.dl0)
        want, v, bound = R.adapter_linear(self.x, self.who, self.A, self.B, self.y0, self.scale)
        _near(self.y, want, bound)
        assert torch.equal(self.y[self.who == self.A.shape[0]], self.y0[self.who == self.A.shape[0]])
        _gradients_near(self.grads, (self.x, self.who, self.A, self.B, self.v, self.dy, self.dx0, self.scale))

    def outputs(self):
        return [t.clone() for t in (self.loss, self.counts, self.y, self.v, self.dl, *self.grads)]


@pytest.mark.parametrize("T,H,N,E,k,rank,n", [(1, 64, 96, 8, 2, 8, 1), (61, 256, 544, 16, 4, 16, 3), (700, 544, 288, 64, 6, 32, 5)])
def test_fine_tuning_step(gpu, T, H, N, E, k, rank, n):
    import torch
    m, dev = gpu
    s = _Step(m, dev, T, H, N, E, k, rank, n, T)
    s.forward()
    s.backward()
    s.check()
    before = [g.clone() for g in s.grads[1:]]
    norm = m.clip_grad_norm(m.GradSet(list(s.grads[1:])), 0.5)
    total = float(torch.stack([g.double().square().sum() for g in before]).sum().sqrt())
    # the FP64 sums of at most 2^17 squares, in another order each
    assert abs(float(norm) - total) <= 2.0 ** -35 * total and total > 0.5
    for b, g in zip(before, s.grads[1:]):
        assert torch.equal(g, (b.double() * (0.5 / float(norm))).float())


def test_captured_fine_tuning_step(gpu):
    """Forward and backward in one graph, replayed with other inputs between eager steps of the same operators."""
    import torch
    m, dev = gpu
    s = _Step(m, dev, 300, 128, 224, 16, 4, 16, 3, 7)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.forward()
        s.backward()
    for _ in range(3):
        s.x.copy_(_randn(s.g, 300, 128))
        s.dy.mul_(-0.5)
        s.who.copy_(torch.randint(-1, 4, (300,), generator=s.g, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        got = s.outputs()
        e = copy.copy(s)
        e.ws = m.adapter_alloc_workspace(300, 128, 224, 16, 3, backward=True, device=dev)
        e.forward()
        e.backward()
        assert all(torch.equal(a, b) for a, b in zip(got, e.outputs()))


@pytest.mark.parametrize("T", [1, 5, 300])
def test_experts_with_adapters(gpu, T):
    """Rows sorted by expert, the experts' products in MXFP4, an adapter per expert on top, and its gradients."""
    import torch
    m, dev = gpu
    H, N, E, k, rank = 192, 160, 12, 3, 16
    g = torch.Generator(device=dev).manual_seed(T)
    W = m.Mxfp4Weights(E, N, H, dev).quantize_from(_randn(g, E, N, H, std=0.1))
    Wt = m.Mxfp4Weights(E, H, N, dev).quantize_from(_randn(g, E, H, N, std=0.1))
    A, B = _randn(g, E, rank, H, std=0.1), _randn(g, E, N, rank, std=0.1)
    x, l = _randn(g, T, H), torch.randn(T, E, generator=g, device=dev)
    ids, _ = m.router_select(l, k)
    loss, counts = m.router_balance_loss(l, ids, 1.0)
    expert, pair = torch.sort(ids.flatten(), stable=True)
    offsets = torch.searchsorted(expert, torch.arange(E + 1, device=dev, dtype=torch.int32)).int()
    assert torch.equal(offsets[1:] - offsets[:-1], counts[0])
    rows = x[pair // k]
    y0 = m.mxfp4_grouped_linear(rows, offsets, W)
    v = torch.empty(T * k, rank, device=dev)
    y = m.adapter_linear(rows, expert, A, B, y0, v=v)
    want, _, bound = R.adapter_linear(rows, expert, A, B, y0, None)
    _near(y, want, bound)
    dy = _randn(g, T * k, N)
    dx0 = m.mxfp4_grouped_linear(dy, offsets, Wt)
    _gradients_near(m.adapter_backward(rows, expert, A, B, v, dy, dx0), (rows, expert, A, B, v, dy, dx0, None))


# --- where the kernels change -------------------------------------------------------------------------

@pytest.mark.parametrize("M,K,N,rank,n", [(512, 72, 136, 16, 2), (513, 72, 136, 16, 2), (512, 136, 72, 64, 40),
                                          (513, 136, 72, 64, 40), (1024, 264, 136, 16, 2), (1025, 264, 136, 16, 2),
                                          (4096, 72, 72, 8, 1), (4097, 72, 72, 8, 1), (3000, 136, 264, 128, 1),
                                          (2000, 520, 72, 32, 1), (9001, 64, 64, 16, 700)])
@pytest.mark.parametrize("order", ["one", "even", "last"])
def test_adapter_boundaries(gpu, M, K, N, rank, n, order):
    """Whole numbers, exact; all rows of one adapter, dealt out in turn, or all but one of the last adapter."""
    import torch
    m, dev = gpu
    g = torch.Generator(device=dev).manual_seed(M + K)

    def ints(*shape, top=1):
        return torch.randint(-top, top + 1, shape, generator=g, device=dev).to(torch.bfloat16)

    ids = torch.zeros(M, dtype=torch.int32, device=dev)
    if order == "even":
        ids.copy_(torch.arange(M, device=dev) % n)
    elif order == "last":
        ids.fill_(n - 1)
        ids[M // 2] = 0
    x, A, B, base, dy, dxb = ints(M, K), ints(n, rank, K), ints(n, N, rank), ints(M, N, top=100), ints(M, N), ints(M, K, top=9)
    scale = 2.0 ** torch.randint(-1, 2, (n,), generator=g, device=dev).float()
    v = torch.empty(M, rank, device=dev)
    got = m.adapter_linear(x, ids, A, B, base, scale, v=v)
    want, wv, _ = R.adapter_linear(x, ids, A, B, base, scale)
    assert torch.equal(got, want.float().to(torch.bfloat16)) and torch.equal(v.double(), wv)
    got = m.adapter_backward(x, ids, A, B, v, dy, dxb, scale)
    want, _ = R.adapter_backward(x, ids, A, B, v, dy, dxb, scale)
    assert float(want[1].abs().max()) < 2 ** 23 and float(want[2].abs().max()) < 2 ** 23
    assert torch.equal(got[0], want[0].float().to(torch.bfloat16))
    assert torch.equal(got[1].double(), want[1]) and torch.equal(got[2].double(), want[2])


@pytest.mark.parametrize("T", [256, 257, 512, 32768, 32769])
def test_balance_boundaries(gpu, T):
    import torch
    m, dev = gpu
    g = torch.Generator(device=dev).manual_seed(T)
    l = torch.randn(T, 24, generator=g, device=dev)
    ids = m.router_select(l, 4)[0]
    add = torch.randn(T, 24, generator=g, device=dev).mul(1e-5)
    for off in (None, [0, 1, T], [0, T - 1, T], [0, 256, T], [3, 255, 256], list(range(0, T + 1, T // 64))):
        o = None if off is None else torch.tensor(off, dtype=torch.int32, device=dev)
        loss, counts = m.router_balance_loss(l, ids, 0.01, offsets=o)
        d = m.router_balance_backward(l, counts, 4, 0.01, offsets=o, add=add)
        _balance_near(m, loss, counts, d, l, ids, 0.01, o, add)


@pytest.mark.parametrize("T", [100, 1000])
def test_many_sequences_without_rows(gpu, T):
    """65536 sequences, of which three have rows: the same as those three alone."""
    import torch
    m, dev = gpu
    S = 65536
    l, ids = torch.randn(T, 40, device=dev), torch.randint(0, 40, (T, 2), device=dev).int()
    off = torch.zeros(S + 1, dtype=torch.int32, device=dev)
    off[2:40000], off[40000:60001], off[60001:] = 10, 60, T
    few = torch.tensor([0, 10, 60, T], dtype=torch.int32, device=dev)
    loss, counts = m.router_balance_loss(l, ids, 0.01, offsets=off)
    want, n = m.router_balance_loss(l, ids, 0.01, offsets=few)
    assert abs(float(loss) - float(want)) <= 2 * 97 * R.U * float(want)
    assert torch.equal(counts[[1, 39999, 60000]], n) and int(counts.sum()) == 2 * T
    got = m.router_balance_backward(l, counts, 2, 0.01, offsets=off)
    assert torch.equal(got, m.router_balance_backward(l, n, 2, 0.01, offsets=few))


def test_decreasing_offsets_stay_in_the_buffers(gpu):
    """The results are undefined, what lies beside the outputs is not."""
    import torch
    m, dev = gpu
    for T in (50, 700):
        l = torch.randn(T, 40, device=dev)
        ids = torch.randint(0, 40, (T, 2), device=dev).int()
        for off in ([0, 40, 10, T], [T, 0], [30, 20, 10, 0], [0, T, 0, T], [2 ** 31 - 1, -2 ** 31, 5, 3]):
            o = torch.tensor(off, dtype=torch.int32, device=dev)
            loss, counts = m.router_balance_loss(l, ids, 0.01, offsets=o)
            buf = torch.full((T + 2, 40), 7.0, device=dev)
            m.router_balance_backward(l, counts, 2, 0.01, offsets=o, out=buf[1:T + 1])
            assert (buf[0] == 7).all() and (buf[-1] == 7).all()
        good = m.router_balance_loss(l, ids, 0.01)
        assert abs(float(good[0]) - R.balance_loss(l, ids, 0.01, False)[0]) < 97 * R.U


@pytest.mark.parametrize("M,K,N,rank,n", [(1, 72, 40, 8, 3), (300, 136, 72, 16, 5), (700, 72, 136, 40, 1024), (2000, 264, 72, 128, 2)])
def test_workspaces_are_kept_to(gpu, M, K, N, rank, n):
    """The workspace may hold anything, and its size is enough: nothing behind it is written."""
    import torch
    m, dev = gpu
    g = torch.Generator(device=dev).manual_seed(M)
    x, A, B, dy = _randn(g, M, K), _randn(g, n, rank, K), _randn(g, n, N, rank), _randn(g, M, N)
    ids = torch.randint(-1, n, (M,), generator=g, device=dev).int()
    results = []
    for fill in (0, 0xFF, 0x5A):
        out = []
        for backward in (False, True):
            size = m.adapter_workspace_bytes(M, K, N, rank, n, backward)
            buf = torch.full((size + 4096,), fill, dtype=torch.uint8, device=dev)
            v = torch.empty(M, rank, device=dev)
            out.append(m.adapter_linear(x, ids, A, B, v=v, workspace=buf[:size]))
            if backward:
                out += m.adapter_backward(x, ids, A, B, v, dy, workspace=buf[:size])
            assert (buf[size:] == fill).all()
        results.append(out)
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


# --- past 32 bits -------------------------------------------------------------------------------------

def test_balance_past_32_bits(gpu):
    import torch
    m, dev = gpu
    T, E = (1 << 24) + 5, 256  # 2^32 + 1280 logits
    l = torch.empty(T, E, dtype=torch.bfloat16, device=dev)
    block = torch.randn(1 << 20, E, device=dev).to(torch.bfloat16)
    for t in range(0, T, 1 << 20):
        l[t:t + (1 << 20)] = block[:min(1 << 20, T - t)]
    ids = torch.randint(0, E, (T, 8), device=dev).int()
    loss, counts = m.router_balance_loss(l, ids, 0.01)
    assert int(counts.sum()) == 8 * T and torch.equal(counts[0].long(), torch.bincount(ids.flatten(), minlength=E))
    off = torch.tensor([T - 37, T], dtype=torch.int32, device=dev)
    loss, counts = m.router_balance_loss(l, ids, 0.01, offsets=off)
    last, few = l[-37:].contiguous(), ids[-37:].contiguous()
    want, n = m.router_balance_loss(last, few, 0.01)
    assert torch.equal(counts, n) and abs(float(loss) - float(want)) <= 2 * 97 * R.U * float(want)
    d = m.router_balance_backward(l, counts, 8, 0.01, offsets=off)
    assert torch.equal(d[-37:], m.router_balance_backward(last, n, 8, 0.01)) and not d[:-37].any()


def test_adapters_past_32_bits(gpu):
    """More than 2^32 elements of x and dx, then of out and dy: the last rows, which alone have the last adapter."""
    import torch
    m, dev = gpu
    M, rank, few = 70001, 16, 19
    for K, N in ((65600, 64), (64, 65600)):
        g = torch.Generator(device=dev).manual_seed(K)
        block = _randn(g, 4096, 65600)
        wide = torch.empty(M, 65600, dtype=torch.bfloat16, device=dev)
        for r in range(0, M, 4096):
            wide[r:r + 4096] = block[:min(4096, M - r)]
        thin = _randn(g, M, 64)
        x, dy = (wide, thin) if K > N else (thin, wide)
        A, B = _randn(g, 2, rank, K, std=0.01), _randn(g, 2, N, rank, std=0.1)
        ids = torch.zeros(M, dtype=torch.int32, device=dev)
        ids[-few:] = 1
        v = torch.empty(M, rank, device=dev)
        y = m.adapter_linear(x, ids, A, B, v=v)
        tail = [t[-few:].contiguous() for t in (x, ids, v, dy)]
        tv = torch.empty(few, rank, device=dev)
        assert torch.equal(y[-few:], m.adapter_linear(tail[0], tail[1], A, B, v=tv)) and torch.equal(v[-few:], tv)
        del y
        dx, dA, dB = m.adapter_backward(x, ids, A, B, v, dy)
        want = m.adapter_backward(tail[0], tail[1], A, B, tail[2], tail[3])
        # (the sums of 19 rows are one step of the same products at any split)
        assert torch.equal(dx[-few:], want[0]) and torch.equal(dA[1], want[1][1]) and torch.equal(dB[1], want[2][1])


def test_adapter_weights_past_32_bits(gpu):
    """A and B of more than 2^32 bytes each: the last adapter, in both forms of the forward pass and in the gradients."""
    import torch
    m, dev = gpu
    n, rank, K = 1024, 128, 17000
    A = torch.zeros(n, rank, K, dtype=torch.bfloat16, device=dev)  # 2.2e9 elements, 4.5 GB
    B = torch.zeros(n, K, rank, dtype=torch.bfloat16, device=dev)
    g = torch.Generator(device=dev).manual_seed(0)
    A[-1], B[-1] = _randn(g, rank, K, std=0.01), _randn(g, K, rank, std=0.1)
    for M in (3, 600):
        x, dy = _randn(g, M, K), _randn(g, M, K)
        ids, zero = torch.full((M,), n - 1, dtype=torch.int32, device=dev), torch.zeros(M, dtype=torch.int32, device=dev)
        v, v1 = torch.empty(M, rank, device=dev), torch.empty(M, rank, device=dev)
        one = (A[-1:].contiguous(), B[-1:].contiguous())
        y = m.adapter_linear(x, ids, A, B, v=v)
        assert torch.equal(y, m.adapter_linear(x, zero, *one, v=v1)) and torch.equal(v, v1) and y.any()
        dx, dA, dB = m.adapter_backward(x, ids, A, B, v, dy)
        want = m.adapter_backward(x, zero, *one, v, dy)
        assert torch.equal(dx, want[0]) and torch.equal(dA[-1:], want[1]) and torch.equal(dB[-1:], want[2])
        assert not dA[:-1].any() and not dB[:-1].any()


# --- streams ------------------------------------------------------------------------------------------

def _calls(m, dev):
    """{name: (inputs, what makes of them a call on a stream)}"""
    import torch
    g = torch.Generator(device=dev).manual_seed(1)
    l, ids = torch.randn(4096, 64, generator=g, device=dev), torch.randint(0, 64, (4096, 4), generator=g, device=dev).int()
    off = torch.tensor([0, 1000, 4096], dtype=torch.int32, device=dev)
    counts, dloss = m.router_balance_loss(l, ids, 0.01, offsets=off)[1], torch.full((1,), 0.5, device=dev)
    x, who = _randn(g, 4096, 256), torch.randint(-1, 3, (4096,), generator=g, device=dev).int()
    A, B, scale, base, dy = _randn(g, 3, 16, 256), _randn(g, 3, 512, 16), torch.rand(3, device=dev), _randn(g, 4096, 512), _randn(g, 4096, 512)
    v = torch.randn(4096, 16, generator=g, device=dev)
    ws = m.adapter_alloc_workspace(4096, 256, 512, 16, 3, backward=True, device=dev)
    return {
        "router_balance_loss": ((l, ids, off), lambda l, i, o: lambda s: m.router_balance_loss(l, i, 0.01, offsets=o, stream=s)),
        "router_balance_backward": ((l, counts, off, dloss, l), lambda l, c, o, d, a: lambda s: m.router_balance_backward(
            l, c, 4, 0.01, offsets=o, dloss=d, add=a, stream=s)),
        "adapter_linear": ((x, who, A, B, base, scale, ws), lambda x, i, A, B, b, sc, ws: lambda s: m.adapter_linear(
            x, i, A, B, b, sc, workspace=ws, stream=s)),
        "adapter_backward": ((x, who, A, B, v, dy, scale, ws), lambda x, i, A, B, v, dy, sc, ws: lambda s: m.adapter_backward(
            x, i, A, B, v, dy, None, sc, workspace=ws, stream=s)),
    }


@pytest.mark.parametrize("name", ["router_balance_loss", "router_balance_backward", "adapter_linear", "adapter_backward"])
def test_memory_of_dropped_tensors_waits_for_the_stream(gpu, name):
    import torch
    m, dev = gpu
    inputs, make = _calls(m, dev)[name]
    want = make(*[t.clone() for t in inputs])(None)
    side = torch.cuda.Stream(dev)
    sizes = [t.numel() * t.element_size() for t in inputs]
    # What is allocated below comes from the caches: an allocation of the driver's may wait for the GPU.
    make(*[t.clone() for t in inputs])(side)
    warm = [torch.empty(n, dtype=torch.uint8, device=dev) for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    mine = [t.clone() for t in inputs]
    call = make(*mine)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000_000)  # about half a second
    got = call(side)
    taken = {t.data_ptr() for t in mine}
    mine = call = warm = None
    new = [torch.empty(n, dtype=torch.uint8, device=dev) for n in sizes for _ in range(3)]
    assert not side.query()  # the call's work still waits, and its memory with it
    assert not taken & {t.data_ptr() for t in new}
    side.synchronize()
    for a, b in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
        assert torch.equal(a, b)


def test_a_named_stream_under_capture(gpu):
    import torch
    m, dev = gpu
    side = torch.cuda.Stream(dev)
    calls = _calls(m, dev)
    for inputs, make in calls.values():
        make(*inputs)(None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = [make(*inputs)(side) for inputs, make in calls.values()]
    for _ in range(3):
        for name, k in (("router_balance_loss", 0), ("adapter_linear", 0)):
            calls[name][0][k].mul_(-1.25)
        g.replay()
        torch.cuda.synchronize()
        mine = [[t.clone() for t in (o if isinstance(o, tuple) else (o,))] for o in got]
        for a, (inputs, make) in zip(mine, calls.values()):
            b = make(*inputs)(None)
            assert all(torch.equal(p, q) for p, q in zip(a, b if isinstance(b, tuple) else (b,)))


def test_empty_tensors_on_a_named_stream(gpu):
    import torch
    m, dev = gpu
    side = torch.cuda.Stream(dev)
    l, ids = torch.empty(0, 16, device=dev), torch.empty(0, 4, dtype=torch.int32, device=dev)
    loss, counts = m.router_balance_loss(l, ids, 0.01, stream=side)
    assert m.router_balance_backward(l, counts, 4, 0.01, stream=side).shape == (0, 16)
    x, who = torch.empty(0, 64, dtype=torch.bfloat16, device=dev), torch.empty(0, dtype=torch.int32, device=dev)
    A, B = torch.ones(2, 8, 64, dtype=torch.bfloat16, device=dev), torch.ones(2, 40, 8, dtype=torch.bfloat16, device=dev)
    y = m.adapter_linear(x, who, A, B, stream=side)
    dx, dA, dB = m.adapter_backward(x, who, A, B, torch.empty(0, 8, device=dev), y, stream=side)
    side.synchronize()
    assert y.shape == (0, 40) and dx.shape == (0, 64) and not dA.any() and not dB.any()
    assert float(loss) == 0.0 and not counts.any()


def test_two_calls_at_once(gpu):
    """The same inputs on two streams at once, each with a workspace of its own."""
    import torch
    m, dev = gpu
    calls = _calls(m, dev)
    want = {k: make(*i)(None) for k, (i, make) in calls.items()}
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    own = [{k: [*i[:-1], i[-1].clone()] if k.startswith("adapter") else i for k, (i, _) in calls.items()} for _ in streams]
    torch.cuda.synchronize()
    got = [[(k, calls[k][1](*own[j][k])(s)) for _ in range(5) for k in calls] for j, s in enumerate(streams)]
    torch.cuda.synchronize()
    for outs in got:
        for k, o in outs:
            for a, b in zip(o if isinstance(o, tuple) else (o,), want[k] if isinstance(want[k], tuple) else (want[k],)):
                assert torch.equal(a, b)


@pytest.mark.parametrize("rank,n,order", [(8, 1, "runs"), (16, 3, "mixed"), (32, 5, "runs"), (64, 3, "mixed"), (64, 200, "mixed"), (128, 2, "runs")])
def test_rows_do_not_depend_on_large_batches(gpu, rank, n, order):
    """Rows of batches that take tiles of either height, whole or shared out by columns, to the bit what they are alone;
    ids that start at any address."""
    import torch
    m, dev = gpu
    M, K, N = 9001, 328, 1544
    g = torch.Generator(device=dev).manual_seed(rank + n)
    x, base, A, B = _randn(g, M, K), _randn(g, M, N), _randn(g, n, rank, K, std=0.05), _randn(g, n, N, rank, std=0.1)
    ids = torch.empty(M + 1, dtype=torch.int32, device=dev)[1:]
    ids.copy_(torch.randint(-1, n, (M,), generator=g, device=dev))
    if order == "runs":
        ids.copy_(ids.sort()[0])
    whole, v = torch.empty_like(base), torch.empty(M, rank, device=dev)
    m.adapter_linear(x, ids, A, B, base, v=v, out=whole)
    for rows in (torch.arange(0, 3), torch.arange(M - 300, M), torch.arange(0, 4200), torch.arange(0, M, 2), torch.arange(1000, 1600),
                 torch.randperm(M, generator=torch.Generator().manual_seed(1))[:8200]):
        i = rows.to(dev)
        vp = torch.empty(len(rows), rank, device=dev)
        part = m.adapter_linear(x[i], ids[i], A, B, base[i], v=vp)
        assert torch.equal(part, whole[i]) and torch.equal(vp, v[i])


@pytest.mark.parametrize("T,E,S", [(256, 128, 4), (256, 128, 5), (256, 129, 1), (64, 512, 4), (65, 512, 2), (16, 1024, 9), (17, 1024, 9),
                                   (33, 1000, 40), (700, 600, 700), (5000, 64, 1500), (9000, 300, 3)])
def test_balance_launches(gpu, T, E, S):
    """Around the sizes of one launch, and workgroups of fewer rows for short sequences; the workspace dirty."""
    import torch
    m, dev = gpu
    g = torch.Generator(device=dev).manual_seed(T + S)
    l = torch.randn(T, E, generator=g, device=dev)
    ids = torch.randint(0, E, (T, 4), generator=g, device=dev).int()
    cut = torch.randint(0, T + 1, (S - 1,), generator=g, device=dev).sort()[0]
    off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)]).int()
    dirty = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=dev)
    del dirty
    loss, counts = m.router_balance_loss(l, ids, 0.01, offsets=off)
    d = m.router_balance_backward(l, counts, 4, 0.01, offsets=off)
    _balance_near(m, loss, counts, d, l, ids, 0.01, off, None)
    for _ in range(3):
        again = m.router_balance_loss(l, ids, 0.01, offsets=off)
        assert torch.equal(again[0], loss) and torch.equal(again[1], counts)


@pytest.mark.parametrize("T,E,S", [(700, 40, 1024), (700, 40, 1025), (3000, 100, 600), (20000, 24, 5000), (300, 8, 65536)])
def test_balance_of_many_sequences(gpu, T, E, S):
    """Most of them short, one of a third of the rows: against sums per sequence in FP64."""
    import torch
    m, dev = gpu
    g = torch.Generator(device=dev).manual_seed(T + S)
    l = torch.randn(T, E, generator=g, device=dev)
    ids = torch.randint(0, E, (T, 2), generator=g, device=dev).int()
    cut = torch.randint(0, T + 1, (S - 1,), generator=g, device=dev).sort()[0]
    cut[(cut > T // 3) & (cut < 2 * T // 3)] = T // 3
    off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)])
    loss, counts = m.router_balance_loss(l, ids, 0.01, offsets=off.int())
    rows = (off[1:] - off[:-1])
    seq = torch.repeat_interleave(torch.arange(S, device=dev), rows)
    n = torch.zeros(S, E, dtype=torch.float64, device=dev).index_put_((seq[:, None].expand(-1, 2), ids.long()), torch.ones((), dtype=torch.float64, device=dev), accumulate=True)
    assert torch.equal(counts.double(), n)
    p = torch.softmax(l.double(), 1)
    f = n * E / (2 * rows[:, None].clamp(min=1))
    want = 0.01 / T * float((f[seq] * p).sum())
    assert abs(float(loss) - want) <= 97 * R.U * want
    d = m.router_balance_backward(l, counts, 2, 0.01, offsets=off.int())
    ref = 0.01 / T * p * (f[seq] - (f[seq] * p).sum(1, keepdim=True))
    # w within 12 u, D^2 within 24, the difference's terms within 12 of their size, and the last rounding
    size = 0.01 / T * p * (f[seq] + (f[seq] * p).sum(1, keepdim=True))
    assert ((d.double() - ref).abs() <= 64 * R.U * size + 1e-36).all()
