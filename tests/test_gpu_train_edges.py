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


@pytest.mark.parametrize("rank", [8, 32, 64, 128])
@pytest.mark.parametrize("M", [2, 600])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_values_stay_finite(gpu, M, rank, sign):
    """v and w between the largest BF16 value and the largest FP32 one, which have no BF16 rounding but infinity:
    outputs and gradients that are finite, whole in FP32, and rounded once."""
    import torch
    m, dev = gpu
    bf, K, N = torch.bfloat16, 72, 136
    top, more, tiny = sign * float(torch.finfo(bf).max), sign * 0.9375 * 2.0 ** 120, 2.0 ** -100
    big = torch.tensor(top, dtype=torch.float64) + more
    assert float(big.float()) == float(big) and torch.isinf(big.to(bf))

    def pair(wide):  # a row of ones, and what makes `big` of it
        x, z = torch.zeros(wide), torch.zeros(rank, wide)
        x[:2], z[rank - 1, :2] = 1.0, torch.tensor([top, more])
        return x.to(bf).to(dev).expand(M, -1).contiguous(), z.to(bf).to(dev)[None].contiguous()

    ids = torch.zeros(M, dtype=torch.int32, device=dev)
    x, A = pair(K)
    B = torch.full((1, N, rank), tiny, dtype=bf, device=dev)
    v = torch.empty(M, rank, device=dev)
    out = m.adapter_linear(x, ids, A, B, v=v)
    assert (v[:, rank - 1].double() == float(big)).all() and not v[:, :rank - 1].any()
    assert torch.equal(out, (big * tiny).float().to(bf).to(dev).expand(M, N))
    # one row of dy is not zero: dB = dy v^T.  (v's own gradients are small: B is.)
    dy = torch.zeros(M, N, dtype=bf, device=dev)
    dy[1] = tiny
    _, _, dB = m.adapter_backward(x, ids, A, B, v, dy)
    assert (dB[0, :, rank - 1].double() == float(big) * tiny).all() and not dB[0, :, :rank - 1].any()
    # w = B^T dy of that size, in one row: dx = A^T w and dA = w x^T
    dy, Bt = pair(N)
    dy[0] = 0
    dy[2:] = 0
    x = torch.full((M, K), tiny, dtype=bf, device=dev)
    A = torch.full((1, rank, K), tiny, dtype=bf, device=dev)
    dx, dA, _ = m.adapter_backward(x, ids, A, Bt.transpose(1, 2).contiguous(), torch.zeros_like(v), dy)
    assert torch.equal(dx[1], (big * tiny).float().to(bf).to(dev).expand(K)) and not dx[0].any() and not dx[2:].any()
    assert (dA[0, rank - 1].double() == float(big) * tiny).all() and not dA[0, :rank - 1].any()


def _milliseconds(f):
    """The shortest of five calls."""
    import torch
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("T", [12, 100, 1000, 16384])
@pytest.mark.parametrize("where", ["before", "between", "behind", "within"])
def test_sequences_without_rows_cost_little(gpu, T, where):
    """65536 sequences of which a few have rows: what those few alone give, in less than 2 ms.  (Well below 0.2 where
    nothing steps through them one by one, which takes 8 to 16.)"""
    import torch
    m, dev = gpu
    S, E, k = 65536, 40, 2
    l, ids = torch.randn(T, E, device=dev), torch.randint(0, E, (T, k), device=dev).int()
    few = torch.tensor([0, 3, 9, T], dtype=torch.int32, device=dev)
    off = torch.empty(S + 1, dtype=torch.int32, device=dev)
    if where == "before":
        at = [S - 3, S - 2, S - 1]
        off[:] = 0
        off[-3:] = few[1:]
    elif where == "between":
        at = [0, 30000, 65000]
        off[:1], off[1:30001], off[30001:65001], off[65001:] = 0, 3, 9, T
    elif where == "behind":
        at = [0, 1, 2]
        off[:] = T
        off[:3] = few[:3]
    else:  # the rows before the first offset and behind the last belong to none
        few = torch.tensor([2, 5, 7, 11], dtype=torch.int32, device=dev)
        at = [40000, 40001, 65535]
        off[:40001], off[40001:40002], off[40002:65536], off[65536:] = 2, 5, 7, 11
    loss, counts = m.router_balance_loss(l, ids, 0.01, offsets=off)
    want, n = m.router_balance_loss(l, ids, 0.01, offsets=few)
    # sums over at most 256 tokens in FP32, then FP64, in chunks of other sizes
    assert abs(float(loss) - float(want)) <= 2 * 97 * 2.0 ** -24 * float(want)
    assert torch.equal(counts[at], n) and int(counts.sum()) == int(n.sum()) == k * int(few[3] - few[0])
    d = m.router_balance_backward(l, counts, k, 0.01, offsets=off)
    assert torch.equal(d, m.router_balance_backward(l, n, k, 0.01, offsets=few))
    assert _milliseconds(lambda: m.router_balance_loss(l, ids, 0.01, offsets=off)) < 2
    assert _milliseconds(lambda: m.router_balance_backward(l, counts, k, 0.01, offsets=off)) < 2


@pytest.mark.parametrize("dloss", [float("inf"), float("-inf"), float("nan")])
def test_a_loss_scale_that_overflowed(gpu, dloss):
    """A gradient of the loss that is not finite: unusable logits, rows masked whole and rows of no sequence still get
    `add` alone (or 0), every other row shows that it overflowed."""
    import torch
    m, dev = gpu
    for E, kind in ((16, torch.float32), (130, torch.bfloat16), (600, torch.float32), (1000, torch.bfloat16)):
        for score in (m.SCORE_SOFTMAX, m.SCORE_SIGMOID):
            l = torch.randn(40, E, device=dev).to(kind)
            l[:, ::3] = -float("inf")
            l[:, 1::7] = float("nan")
            l[5] = -float("inf")
            ids = torch.randint(0, E, (40, 2), device=dev).int()
            ids[:, 0] = 2
            off = torch.tensor([3, 20, 37], dtype=torch.int32, device=dev)
            add = torch.randn(40, E, device=dev).to(kind)
            _, counts = m.router_balance_loss(l, ids, 0.01, score=score, offsets=off)
            scale = torch.full((1,), dloss, device=dev)
            dead = ~(l > -float("inf"))
            dead[:3] = dead[37:] = True
            for a in (add, None):
                d = m.router_balance_backward(l, counts, 2, 0.01, score=score, offsets=off, dloss=scale, add=a)
                assert torch.equal(d[dead], add[dead] if a is not None else torch.zeros_like(add[dead]))
                live = ~dead.all(1)
                assert (~torch.isfinite(d[live])).any(1).all()


def test_balance_of_2_to_the_30_rows(gpu):
    """More chunks than a launch has workgroups along one axis.  Rows repeat every 2^20."""
    import torch
    m, dev = gpu
    P, times, rest = 1 << 20, 1024, 5
    T, E = P * times + rest, 2
    few = torch.randn(P, E, device=dev).to(torch.bfloat16)
    one = torch.randint(0, E, (P, 1), device=dev).int()
    l, ids = torch.empty(T, E, dtype=torch.bfloat16, device=dev), torch.empty(T, 1, dtype=torch.int32, device=dev)
    for t in range(0, T, P):
        l[t:t + P], ids[t:t + P] = few[:T - t], one[:T - t]
    p = torch.softmax(few.double(), 1)
    for cut in (None, P * 1000 + 3):
        # (times, rest) of each sequence, and where its rows begin in the pattern
        parts = [(0, T)] if cut is None else [(0, cut), (cut, T)]
        off = None if cut is None else torch.tensor([0, cut, T], dtype=torch.int32, device=dev)
        loss, counts = m.router_balance_loss(l, ids, 1.0, offsets=off)
        d = m.router_balance_backward(l, counts, 1, 1.0, offsets=off)
        want = 0.0

        def upto(x, n):  # the sum of the first n rows of the repeated x
            return x.sum(0) * (n // P) + x[:n % P].sum(0)

        hot = torch.nn.functional.one_hot(one[:, 0].long(), E)
        for s, (a, b) in enumerate(parts):
            n = upto(hot, b) - upto(hot, a)
            assert torch.equal(counts[s].long(), n)
            f = n.double() * E / (b - a)
            want += float((f * (upto(p, b) - upto(p, a))).sum()) / T
            for r in (a, b - 37):  # some of the sequence's rows
                q = p[torch.arange(r, r + 37, device=dev) % P]
                ref = q * (f - (q @ f[:, None])) / T
                # every term within 64 u of its size, then the rounding to BF16
                size = q * (f + (q @ f[:, None])) / T
                assert ((d[r:r + 37].double() - ref).abs() <= 64 * 2.0 ** -24 * size + 2.0 ** -8 * ref.abs() + 1e-38).all()
        assert abs(float(loss) - want) <= 97 * 2.0 ** -24 * want
        del d


# --- branches that only large calls reach -------------------------------------------------------------

def _ints(g, *shape, top=1):
    import torch
    return torch.randint(-top, top + 1, shape, generator=g, device=g.device).to(torch.bfloat16)


@pytest.mark.parametrize("M,n,rank", [((1 << 18) + 77, 37, 16), (600001, 1000, 8), (600001, 3, 24)])
@pytest.mark.parametrize("order", ["mixed", "sorted"])
def test_adapters_of_more_rows_than_the_plan_has_threads(gpu, M, n, rank, order):
    """A workgroup of the plan places several times 1024 rows from 2^18 on.  Whole numbers, exact."""
    import torch
    from tests import plain_train_ops as R
    m, dev = gpu
    g = torch.Generator(device=dev).manual_seed(M + n)
    K, N = 64, 72
    x, A, B, dy = _ints(g, M, K), _ints(g, n, rank, K), _ints(g, n, N, rank), _ints(g, M, N)
    base, dxb = _ints(g, M, N, top=100), _ints(g, M, K, top=9)
    ids = torch.randint(-1, n + 1, (M,), generator=g, device=dev).int()
    if order == "sorted":
        ids = ids.sort()[0]
    v = torch.empty(M, rank, device=dev)
    got = m.adapter_linear(x, ids, A, B, base, v=v)
    want, wv, _ = R.adapter_linear(x, ids, A, B, base, None)
    assert torch.equal(got, want.float().to(torch.bfloat16)) and torch.equal(v.double(), wv)
    got = m.adapter_backward(x, ids, A, B, v, dy, dxb)
    want, _ = R.adapter_backward(x, ids, A, B, v, dy, dxb, None)
    assert float(want[1].abs().max()) < 2 ** 23 and float(want[2].abs().max()) < 2 ** 23
    assert torch.equal(got[0], want[0].float().to(torch.bfloat16))
    assert torch.equal(got[1].double(), want[1]) and torch.equal(got[2].double(), want[2])


@pytest.mark.parametrize("K,N", [(64, 4096), (4096, 64), (72, 4104)])
@pytest.mark.parametrize("rank", [16, 32, 64, 128])
def test_base_past_the_last_level_cache(gpu, K, N, rank):
    """More than 2^28 bytes of rows, from which on base is read past the cache: beside the output and in place, forward
    and dx.  Whole numbers, exact."""
    import torch
    from tests import plain_train_ops as R
    m, dev = gpu
    M, n = 20011, 5
    assert 2 * M * (min(K, N) + max(K, N)) * 2 >= 1 << 28
    g = torch.Generator(device=dev).manual_seed(rank + K)
    x, A, B, dy = _ints(g, M, K), _ints(g, n, rank, K), _ints(g, n, N, rank), _ints(g, M, N)
    base, dxb = _ints(g, M, N, top=100), _ints(g, M, K, top=9)
    ids = torch.randint(-1, n, (M,), generator=g, device=dev).int()
    v = torch.empty(M, rank, device=dev)
    want = R.adapter_linear(x, ids, A, B, base, None)[0].float().to(torch.bfloat16)
    keep = base.clone()
    assert torch.equal(m.adapter_linear(x, ids, A, B, base, v=v), want) and torch.equal(base, keep)
    m.adapter_linear(x, ids, A, B, base, out=base)
    assert torch.equal(base, want)
    wx, wA, wB = R.adapter_backward(x, ids, A, B, v, dy, dxb, None)[0]
    assert float(wx.abs().max()) < 2 ** 23 and float(wA.abs().max()) < 2 ** 23 and float(wB.abs().max()) < 2 ** 23
    keep = dxb.clone()
    dx, dA, dB = m.adapter_backward(x, ids, A, B, v, dy, dxb)
    wx = wx.float().to(torch.bfloat16)
    assert torch.equal(dx, wx) and torch.equal(dA.double(), wA) and torch.equal(dB.double(), wB) and torch.equal(dxb, keep)
    dx, _, _ = m.adapter_backward(x, ids, A, B, v, dy, dxb, out=(dxb, torch.empty_like(dA), torch.empty_like(dB)))
    assert dx is dxb and torch.equal(dx, wx)


# --- the balance loss's workspace and the neighbours of its outputs -----------------------------------

def _guarded_loss(m, l, ids, off, fill):
    """(loss, counts) through the C entry point, with a workspace of exactly the size that it asks for and outputs that
    are slices; everything filled with `fill` before, and what lies around them checked after."""
    import ctypes
    import torch
    T, E = l.shape
    S = off.numel() - 1

    def slab(size):  # a slice in the middle, 256-byte aligned, and its neighbours
        buf = torch.full((size + 8192,), fill, dtype=torch.uint8, device=l.device)
        return buf[4096:4096 + size], (buf[:4096], buf[4096 + size:])

    need = m.lib().nvfp4moe_balance_workspace_bytes(T, E, S)
    parts = [slab(n) for n in (need, 4, 4 * S * E)]
    ws, loss, counts = (p[0] for p in parts)
    cfg = m.BalanceConfig(E, ids.shape[1], m.SCORE_SOFTMAX, m.F32, 0.01)
    st = m.lib().nvfp4moe_router_balance_loss(ctypes.byref(cfg), l.data_ptr(), l.stride(0), T, ids.data_ptr(), off.data_ptr(), S,
                                              loss.data_ptr(), counts.data_ptr(), ws.data_ptr(), need,
                                              torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for _, around in parts:
        assert all((t == fill).all() for t in around)
    return loss.view(torch.float32).clone(), counts.view(torch.int32).view(S, E).clone()


@pytest.mark.parametrize("T,E,S", [(256, 128, 4), (256, 128, 5), (256, 129, 1), (64, 512, 4), (65, 512, 2), (16, 1024, 9), (17, 1024, 9),
                                   (33, 1000, 40), (700, 600, 700), (5000, 64, 1500), (9000, 300, 3), (700, 40, 1025),
                                   (20000, 24, 5000), (300, 8, 65536), (131073, 16, 2), (50, 33, 200)])
def test_balance_workspace_is_kept_to(gpu, T, E, S):
    """The workspace may hold anything, its size is enough, and the outputs' neighbours stay."""
    import torch
    m, dev = gpu
    g = torch.Generator(device=dev).manual_seed(T + S)
    l = torch.randn(T, E, generator=g, device=dev)
    ids = torch.randint(0, E, (T, 4), generator=g, device=dev).int()
    cut = torch.randint(0, T + 1, (S - 1,), generator=g, device=dev).sort()[0]
    off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)]).int()
    loss, counts = m.router_balance_loss(l, ids, 0.01, offsets=off)
    assert torch.isfinite(loss).all() and int(counts.sum()) == 4 * T
    for fill in (0, 0xFF, 0x5A):
        got = _guarded_loss(m, l, ids, off, fill)
        assert torch.equal(got[0], loss) and torch.equal(got[1], counts)


@pytest.mark.parametrize("T", [50, 700, 5000])
def test_decreasing_offsets_keep_to_the_workspace(gpu, T):
    """The results are undefined, what lies beside loss, counts and workspace is not."""
    import torch
    m, dev = gpu
    l, ids = torch.randn(T, 40, device=dev), torch.randint(0, 40, (T, 2), device=dev).int()
    lists = [[0, 40, 10, T], [T, 0], [30, 20, 10, 0], [0, T, 0, T], [2 ** 31 - 1, -2 ** 31, 5, 3], [5, 5, 3, 3, T, T, 2, 2, T],
             list(range(T, -1, -1)), [T, 0] * 400, [0] * 300 + [T] * 300 + [0] * 300 + [T]]
    for off in lists:
        o = torch.tensor(off, dtype=torch.int32, device=dev)
        for fill in (0xFF, 0x5A):
            counts = _guarded_loss(m, l, ids, o, fill)[1]
            buf = torch.full((T + 2, 40), 7.0, device=dev)
            m.router_balance_backward(l, counts, 2, 0.01, offsets=o, out=buf[1:T + 1])
            assert (buf[0] == 7).all() and (buf[-1] == 7).all()
