"""GPU expert selection (nvfp4moe_router_select) and its gradient against the FP64 plain forms of tests/plain_ops.py.

Bars: ids equal.  probs: formed in FP64 and rounded once, half a step of FP32 (2^-24 relative).  Gradients: one rounding
of an FP64 value (in BF16 a second one).  The first tests allow the softmax over all experts what FP32 terms would need:
three roundings in each exponent (3 x 2^-24 |x|, which over a softmax's terms sums to at most 3 ln E <= 21 steps of
2^-24), one step (2) of the exponential, at most 22 additions: 48 x 2^-24 on each of the two terms of a gradient (and
3 |l - max| more on the one whose exponential is its own); the last ones hold it to FP64."""
import numpy as np
import pytest

import moe_workloads as W
from tests import plain_ops as R
from tests.helpers import to_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_moe_expert_sort_amd as m
    m.lib()
    return m, torch.device("cuda:0")


def _logits(rng, T, E, bf16, std=1.5):
    import torch
    l = torch.from_numpy((rng.standard_normal((T, E)) * std).astype(np.float32))
    return l.to(torch.bfloat16) if bf16 else l


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _select(m, l, k, bias=None, **kw):
    """The library's answer and the plain one; kw as the plain form names them."""
    ids, probs = m.router_select(l, k, bias=bias, score=1 if kw.get("sigmoid") else 0, renormalize=kw.get("renorm", True),
                                 scale=kw.get("scale", 1.0), n_groups=kw.get("n_groups", 1),
                                 top_groups=kw.get("top_groups", 1), group_score=1 if kw.get("top2") else 0)
    b = None if bias is None else _np(bias)
    ref = [R.select_row(row, k, bias=b, **kw) for row in _np(l)]
    return ids.cpu().numpy(), probs.cpu().numpy(), ref


def _check(m, l, k, bias=None, **kw):
    ids, probs, ref = _select(m, l, k, bias, **kw)
    fp32_sum = not kw.get("sigmoid") and not kw.get("renorm", True) and bias is None and not kw.get("top2")
    tol = 48 * U if fp32_sum else 1.01 * U
    for t, (i, p) in enumerate(ref):
        assert ids[t].tolist() == i.tolist(), (t, ids[t], i)
        assert (np.abs(probs[t] - p) <= tol * np.abs(p) + 2.0 ** -149).all(), (t, probs[t], p)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (7, 3), (60, 4), (64, 16), (65, 8), (128, 8), (130, 9), (256, 8), (255, 16),
                                 (256, 17), (300, 8), (384, 32), (512, 8), (1000, 7), (1024, 32)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_select_sizes(gpu, E, k, sigmoid):
    m, dev = gpu
    rng = np.random.default_rng(E * 100 + k)
    for T, renorm, bf16, biased in ((1, True, False, False), (3, False, True, False), (37, True, True, True),
                                    (17, False, False, True)):
        bias = to_dev((rng.standard_normal(E) * 0.1).astype(np.float32), dev) if biased else None
        _check(m, _logits(rng, T, E, bf16).to(dev), k, bias, sigmoid=sigmoid, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("E,G,TG,k", [(8, 8, 3, 3), (16, 2, 1, 8), (60, 5, 2, 12), (64, 64, 20, 8), (96, 3, 2, 6),
                                      (128, 16, 1, 8), (256, 8, 4, 8), (256, 32, 5, 8), (320, 64, 9, 32), (1024, 8, 2, 8),
                                      (1008, 48, 7, 11)])
@pytest.mark.parametrize("top2", [False, True])
def test_select_groups(gpu, E, G, TG, k, top2):
    m, dev = gpu
    rng = np.random.default_rng(E + G)
    for sigmoid in (False, True):
        for biased in (False, True):
            bias = to_dev((rng.standard_normal(E) * 0.1).astype(np.float32), dev) if biased else None
            _check(m, _logits(rng, 29, E, False).to(dev), k, bias, sigmoid=sigmoid, n_groups=G, top_groups=TG, top2=top2)


def test_select_ties_go_to_the_lower_id(gpu):
    import torch
    m, dev = gpu
    rng = np.random.default_rng(3)
    for E in (24, 200, 600):  # few distinct values: many ties, among experts and among groups
        l = torch.from_numpy(rng.integers(0, 3, (40, E)).astype(np.float32)).to(dev)
        zero = torch.zeros(E, device=dev)
        for kw in (dict(), dict(sigmoid=True), dict(n_groups=8, top_groups=3), dict(n_groups=8, top_groups=3, top2=True)):
            for bias in (None, zero):
                _check(m, l, 6, bias, **kw)
    l = torch.tensor([[0.0, -0.0, 0.0, -0.0]], device=dev)
    assert m.router_select(l, 4)[0].tolist() == [[0, 1, 2, 3]]


SPECIAL = [np.nan, -np.inf, np.inf, R.FLT_MAX, -R.FLT_MAX, 0.0, -0.0, 1e-45, -1e-45, 88.0, -120.0, -800.0, 1e30]


@pytest.mark.parametrize("kw", [dict(), dict(renorm=False), dict(sigmoid=True), dict(sigmoid=True, renorm=False),
                                dict(n_groups=4, top_groups=2), dict(sigmoid=True, n_groups=4, top_groups=2, top2=True)])
@pytest.mark.parametrize("biased", [False, True])
def test_select_special_values(gpu, kw, biased):
    import torch
    m, dev = gpu
    rng = np.random.default_rng(11)
    E = 20
    rows = [np.full(E, v) for v in SPECIAL]
    for _ in range(60):
        r = rng.standard_normal(E)
        hit = rng.random(E) < rng.choice([0.2, 0.7])
        r[hit] = rng.choice(SPECIAL, hit.sum())
        rows.append(r)
    l = torch.from_numpy(np.array(rows).astype(np.float32)).to(dev)
    bias = None
    if biased:
        b = rng.standard_normal(E).astype(np.float32) * 0.1
        b[[2, 5, 9, 15]] = [np.nan, -np.inf, np.inf, -R.FLT_MAX]
        bias = torch.from_numpy(b).to(dev)
    ids, probs, ref = _select(m, l, 8, bias, **kw)
    for t, (i, p) in enumerate(ref):
        assert ids[t].tolist() == i.tolist(), (t, rows[t], ids[t], i)
        # e^x of huge and tiny arguments: FP32 results below its normal range are off by their own step
        assert (np.abs(probs[t] - p) <= 48 * U * np.abs(p) + 2.0 ** -149).all(), (t, probs[t], p)
    assert np.isfinite(probs).all()


def test_select_masked_rows_and_low_masks(gpu):
    """Masks of -inf and of the type's lowest value; a row masked whole gives experts 0..k-1 with probability 0."""
    import torch
    m, dev = gpu
    l = torch.randn(6, 32, device=dev)
    l[0] = -torch.inf
    l[1, 4:] = -torch.inf
    l[2, 1:] = torch.finfo(torch.float32).min
    ids, probs = m.router_select(l, 6)
    assert ids[0].tolist() == list(range(6)) and probs[0].tolist() == [0.0] * 6
    assert sorted(ids[1].tolist()[:4]) == [0, 1, 2, 3] and ids[1].tolist()[4:] == [4, 5] and probs[1, 4:].tolist() == [0, 0]
    assert ids[2].tolist() == [0, 1, 2, 3, 4, 5] and probs[2].tolist() == [1.0, 0, 0, 0, 0, 0]
    low = l.to(torch.bfloat16)
    low[3] = torch.finfo(torch.bfloat16).min
    ids, probs = m.router_select(low, 4)
    assert ids[3].tolist() == [0, 1, 2, 3] and probs[3].tolist() == [0.25] * 4


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_select_scores_that_vanish_tie(gpu, sigmoid, biased):
    """A score that FP64 cannot hold is 0: of groups whose experts are masked with the lowest value, one with a single
    usable expert ties with one that has two, and so the lower group stays."""
    m, dev = gpu
    rng = np.random.default_rng(12)
    T, E, G = 24, 64, 16
    l = rng.standard_normal((T, E)).astype(np.float32).reshape(T, G, 4)
    low = rng.random((T, G)) < 0.7
    for value in (-R.FLT_MAX, -2000.0):
        a = np.where(low[..., None], np.float32(value), l)
        a[rng.random(a.shape) < 0.4] = -np.inf
        a = a.reshape(T, E)
        bias = to_dev(np.zeros(E, np.float32), dev) if biased else None
        for renorm in (False, True):
            _check(m, to_dev(a.astype(np.float32), dev), 9, bias, sigmoid=sigmoid, renorm=renorm, n_groups=G, top_groups=9,
                   top2=True)


def test_select_signaling_nan(gpu):
    """Signaling NaN patterns are NaN too."""
    import torch
    m, dev = gpu
    l = torch.randn(5, 70, device=dev)
    quiet = l.clone()
    for t, e in ((0, 3), (1, 69), (2, 0), (4, 33)):
        l.view(torch.int32)[t, e] = 0x7F800001 if t % 2 else -0x7FFFFF  # 0xFF800001
        quiet[t, e] = torch.nan
    bias = torch.zeros(70, device=dev)
    bias.view(torch.int32)[5] = 0x7F800100
    qb = bias.clone()
    qb[5] = torch.nan
    for kw, qw in ((dict(), dict()), (dict(bias=bias), dict(bias=qb)), (dict(score=1, renormalize=False),) * 2):
        a, b = m.router_select(l, 6, **kw), m.router_select(quiet, 6, **qw)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert 5 not in m.router_select(l, 6, bias=bias)[0].flatten().tolist()


def test_select_strides_alignment_and_untouched_neighbours(gpu):
    import torch
    m, dev = gpu
    rng = np.random.default_rng(5)
    for dtype in (torch.float32, torch.bfloat16):
        big = torch.from_numpy(rng.standard_normal((50, 140)).astype(np.float32)).to(dev).to(dtype)
        for c0, E in ((0, 128), (1, 128), (3, 101), (4, 136), (0, 140)):
            l = big[:, c0:c0 + E]
            ids, probs = m.router_select(l, 8)
            a, b = m.router_select(l.contiguous(), 8)
            assert torch.equal(ids, a) and torch.equal(probs, b)
            dp = torch.from_numpy(rng.standard_normal((50, 8)).astype(np.float32)).to(dev)
            wide = torch.full((52, 150), 7.0, device=dev, dtype=dtype)
            out = wide[1:51, c0 + 2:c0 + 2 + E]
            m.router_select_backward(l, ids, dp, renormalize=False, out=out)
            assert torch.equal(out, m.router_select_backward(l.contiguous(), ids, dp, renormalize=False))
            wide[1:51, c0 + 2:c0 + 2 + E] = 7.0
            assert (wide == 7.0).all()


def test_select_is_the_routers_top_k(gpu):
    """Softmax without bias or groups is nvfp4moe_router_topk's selection, on the logits of nvfp4moe_router_logits."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(8)
    x = to_dev(W.f32_to_bf16_bits(rng.standard_normal((77, 256)).astype(np.float32)), dev)
    w = to_dev(W.f32_to_bf16_bits((rng.standard_normal((100, 256)) * 0.05).astype(np.float32)), dev)
    logits, ids, probs = m.router_topk(x, w, 8)
    assert torch.equal(logits, m.router_logits(x, w))
    got, p = m.router_select(logits, 8)
    assert torch.equal(got, ids)
    assert ((p - probs).abs() <= 24 * U * probs).all()  # router_topk forms its softmax in FP32


def test_select_batch_invariance(gpu):
    import torch
    m, dev = gpu
    rng = np.random.default_rng(9)
    l = _logits(rng, 200, 256, False).to(dev)
    bias = torch.randn(256, device=dev) * 0.05
    kw = dict(bias=bias, score=1, n_groups=8, top_groups=4, group_score=1, scale=2.5)
    ids, probs = m.router_select(l, 8, **kw)
    dp = torch.randn(200, 8, device=dev)
    for renorm in (False, True):
        g = m.router_select_backward(l, ids, dp, renormalize=renorm)
        for t0, t1 in ((0, 1), (3, 4), (7, 24), (199, 200)):
            a, b = m.router_select(l[t0:t1], 8, **kw)
            assert torch.equal(a, ids[t0:t1]) and torch.equal(b, probs[t0:t1])
            assert torch.equal(m.router_select_backward(l[t0:t1], ids[t0:t1], dp[t0:t1], renormalize=renorm), g[t0:t1])


def _check_backward(m, dev, l, ids, dp, bias=None, sigmoid=False, renorm=True, scale=1.0):
    import torch
    got = m.router_select_backward(l, torch.from_numpy(ids.astype(np.int32)).to(dev), torch.from_numpy(dp).to(dev),
                                   bias=bias, score=1 if sigmoid else 0, renormalize=renorm, scale=scale)
    assert got.dtype == l.dtype
    rnd = U if l.dtype == torch.float32 else 2.0 ** -8
    b = None if bias is None else _np(bias)
    dense = not sigmoid and not renorm
    for t, row in enumerate(_np(l)):
        ref = R.select_backward_row(row, ids[t], dp[t], bias=b, sigmoid=sigmoid, renorm=renorm, scale=scale)
        size = abs(scale) * np.abs(dp[t]).max()  # FP64 cancellation in dp - mean, and sums of repeated slots
        tol = rnd * np.abs(ref) + 2.0 ** -45 * size + 2.0 ** -149
        slots = np.zeros(len(row))
        for i, d in zip(ids[t], dp[t]):  # one rounding a slot
            if 0 <= i < len(row):
                slots[i] += abs(scale * d)
        if dense:
            usable, c = R.usable_logits(row)
            s = R.scores(c, usable, False)
            far = np.where(usable, np.minimum(np.where(usable, c[usable].max() - c, 0.0) if usable.any() else 0.0, 200.0), 0.0)
            tol = tol + U * s * (50 * slots + (54 + 3 * far) * size * len(ids[t]))
        else:
            tol = tol + (3 * U * slots if len(set(ids[t])) < len(ids[t]) else 0.0)
        g = _np(got[t])
        assert (np.abs(g - ref) <= tol).all(), (t, np.abs(g - ref).max(), np.argmax(np.abs(g - ref) - tol))


@pytest.mark.parametrize("E,k", [(1, 1), (7, 3), (64, 8), (66, 5), (128, 8), (256, 16), (256, 20), (400, 8), (1023, 32)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_select_backward(gpu, E, k, sigmoid, renorm):
    m, dev = gpu
    rng = np.random.default_rng(E + k)
    for T, bf16 in ((1, False), (21, True), (33, False)):
        l = _logits(rng, T, E, bf16).to(dev)
        ids = m.router_select(l, k)[0].cpu().numpy()
        dp = rng.standard_normal((T, k)).astype(np.float32)
        _check_backward(m, dev, l, ids, dp, sigmoid=sigmoid, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_select_backward_odd_ids_and_masks(gpu, sigmoid, renorm):
    """Repeated ids, ids outside [0, E), masked experts, masked rows, an unavailable bias."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(2)
    l = _logits(rng, 40, 50, False).to(dev)
    l[3] = -torch.inf
    l[4, ::2] = -torch.inf
    l[5, 1::2] = torch.nan
    l[6] = -300.0  # sigmoid's terms vanish in FP32, their ratio does not
    ids = rng.integers(0, 50, (40, 6))
    ids[10] = [1, 1, 1, 2, 2, 3]
    ids[11] = [-1, 50, 1 << 30, -(1 << 31), 7, 7]
    ids[12] = -1
    dp = rng.standard_normal((40, 6)).astype(np.float32)
    bias = torch.zeros(50, device=dev)
    bias[[1, 8, 9]] = torch.tensor([-torch.inf, torch.nan, torch.inf], device=dev)
    for b in (None, bias):
        _check_backward(m, dev, l, ids, dp, bias=b, sigmoid=sigmoid, renorm=renorm)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_select_backward_against_differences(gpu, sigmoid, renorm):
    """Central differences of the plain forward in FP64 (error h^2 |f'''| / 6 < 1e-9 and 1e-16 / h)."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(6)
    l = rng.standard_normal((3, 12)).astype(np.float32)
    dp = rng.standard_normal((3, 4)).astype(np.float32)
    dl = torch.from_numpy(l).to(dev)
    ids, _ = m.router_select(dl, 4, score=1 if sigmoid else 0, renormalize=renorm, scale=1.5)
    got = m.router_select_backward(dl, ids, torch.from_numpy(dp).to(dev), score=1 if sigmoid else 0, renormalize=renorm,
                                   scale=1.5).cpu().numpy()
    h = 1e-5
    for t in range(3):
        i = ids[t].cpu().numpy()

        def f(x):
            u, c = R.usable_logits(x)
            return 1.5 * (R.weights(c[i], u[i], sigmoid, renorm, R.scores(c, u, sigmoid)[i]) * dp[t]).sum()

        num = np.array([(f(l[t] + h * e) - f(l[t] - h * e)) / (2 * h) for e in np.eye(12)])
        assert np.abs(got[t] - num).max() < 2e-9 + 60 * U * 1.5 * np.abs(dp[t]).sum()


def test_select_empty_and_outputs(gpu):
    import torch
    m, dev = gpu
    l = torch.empty(0, 16, device=dev)
    ids, probs = m.router_select(l, 4)
    assert ids.shape == probs.shape == (0, 4)
    assert m.router_select_backward(l, ids, probs).shape == (0, 16)
    l = torch.randn(3, 16, device=dev)
    for bad in ((torch.empty(3, 4, dtype=torch.int64, device=dev), torch.empty(3, 4, device=dev)),
                (torch.empty(3, 5, dtype=torch.int32, device=dev), torch.empty(3, 4, device=dev)),
                (torch.empty(3, 4, dtype=torch.int32, device=dev), torch.empty(3, 4, device=dev, dtype=torch.float64))):
        with pytest.raises(ValueError):
            m.router_select(l, 4, out=bad)
    with pytest.raises(ValueError):
        m.router_select_backward(l, torch.zeros(3, 4, dtype=torch.int32, device=dev), torch.zeros(3, 4, device=dev),
                                 out=torch.empty(3, 16, device=dev, dtype=torch.bfloat16))
    with pytest.raises(m.Nvfp4Error):
        m.router_select(l, 17)
    with pytest.raises(m.Nvfp4Error):
        m.router_select(l[:1].expand(3, 16), 4)  # rows on top of each other


def test_select_on_a_side_stream_and_in_a_graph(gpu):
    import torch
    m, dev = gpu
    rng = np.random.default_rng(12)
    l = _logits(rng, 100, 128, False).to(dev)
    dp = torch.randn(100, 8, device=dev)
    want = m.router_select(l, 8)
    back = m.router_select_backward(l, want[0], dp)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream())
    got = m.router_select(l, 8, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = (torch.empty_like(want[0]), torch.empty_like(want[1]))
    dl = torch.empty_like(l)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.router_select(l, 8, out=out)
        m.router_select_backward(l, out[0], dp, out=dl)
    for seed in range(3):
        l.copy_(_logits(np.random.default_rng(seed), 100, 128, False))
        g.replay()
        torch.cuda.synchronize()
        want = m.router_select(l, 8)
        back = m.router_select_backward(l, want[0], dp)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(dl, back)


@pytest.mark.parametrize("E,k", [(5, 3), (128, 8), (256, 8), (256, 20), (700, 8)])
@pytest.mark.parametrize("std", [0.5, 4.0, 30.0])
def test_select_softmax_over_all_is_formed_in_fp64(gpu, E, k, std):
    """Weights without renormalisation: one rounding of an FP64 value (scores within 2^-43, so 1.01 x 2^-24), and the
    same bits with a bias of zero."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(E + k)
    for bf16 in (False, True):
        l = _logits(rng, 57, E, bf16, std).to(dev)
        l[5] = -torch.inf
        l[6, ::3] = -torch.inf
        for groups in (dict(), dict(n_groups=4, top_groups=1)) if E % 4 == 0 else (dict(),):
            ids, probs, ref = _select(m, l, k, renorm=False, **groups)
            for t, (i, p) in enumerate(ref):
                assert ids[t].tolist() == i.tolist()
                assert (np.abs(probs[t] - p) <= 1.01 * U * np.abs(p) + 2.0 ** -149).all(), (t, probs[t], p)
            zero = m.router_select(l, k, bias=torch.zeros(E, device=dev), renormalize=False, **groups)
            assert np.array_equal(zero[1].cpu().numpy(), probs)


@pytest.mark.parametrize("E,k", [(7, 3), (128, 8), (250, 16), (250, 20), (600, 8)])
@pytest.mark.parametrize("gap", [0.0, 5.0, 12.0, 20.0, 34.0])
def test_select_backward_of_confident_tokens(gpu, E, k, gap):
    """Softmax over all experts with one logit `gap` above the others: s_e (dp_e - mean) vanishes as 1 - s does, and is
    formed in FP64.  With r = 1 - max s, the mean is off by some 2^-50 of the largest dp for the top weight and by
    2^-45 r of it for the others (the exponential's 2^-46), so at expert e the bar is one rounding and
    s_e (2^-49 + 2^-44 r) sum |dp|.  With repeated ids too."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(E + int(gap))
    for bf16 in (False, True):
        l = _logits(rng, 40, E, False, 1.0)
        l[torch.arange(40), torch.from_numpy(rng.integers(0, E, 40))] += gap
        l = (l.to(torch.bfloat16) if bf16 else l).to(dev)
        ids = m.router_select(l, k)[0].cpu().numpy()
        ids[30:, 1] = ids[30:, 0]
        dp = rng.standard_normal((40, k)).astype(np.float32)
        got = _np(m.router_select_backward(l, torch.from_numpy(ids).to(dev), torch.from_numpy(dp).to(dev), renormalize=False,
                                           scale=2.5))
        rnd, step = (2.0 ** -8, 2.0 ** -133) if bf16 else (1.01 * U, 2.0 ** -149)
        for t, row in enumerate(_np(l)):
            ref = R.select_backward_row(row, ids[t], dp[t], renorm=False, scale=2.5)
            s = R.scores(row, np.ones(E, bool), False)
            tol = rnd * np.abs(ref) + 2.5 * s * np.abs(dp[t]).sum() * (2.0 ** -49 + 2.0 ** -44 * (1 - s.max())) + step
            assert (np.abs(got[t] - ref) <= tol).all(), (t, np.abs(got[t] - ref).max(), ref[ids[t]])
