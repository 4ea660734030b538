"""The entry points beside the expert forward, without a GPU: refusals on the host (no launch), size functions, the
gradient plan's table, and the plain forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

from tests import plain_ops as R

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
NULL, SHAPE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 9


@pytest.fixture(scope="module")
def m():
    import os
    import nvfp4_moe_expert_sort_amd as m
    if not os.path.exists(m.LIB_PATH):
        from nvfp4_moe_expert_sort_amd import build
        build.build()
    m.lib()
    return m


def _cfg(m, **kw):
    base = dict(n_experts=128, top_k=8, score=0, renormalize=1, scale=1.0, n_groups=1, top_groups=1, group_score=0,
                logits_type=0)
    base.update(kw)
    return m.SelectConfig(*base.values())


@pytest.mark.parametrize("bad,status", [
    (dict(score=2), ARG), (dict(renormalize=2), ARG), (dict(group_score=-1), ARG), (dict(logits_type=2), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(n_experts=0), SHAPE),
    (dict(n_experts=1025), SHAPE), (dict(top_k=0), SHAPE), (dict(top_k=33), SHAPE), (dict(top_k=9, n_experts=8), SHAPE),
    (dict(n_groups=3), SHAPE), (dict(n_groups=128), SHAPE), (dict(n_groups=0), SHAPE),
    (dict(n_groups=4, top_groups=5), SHAPE), (dict(n_groups=4, top_groups=0), SHAPE),
    (dict(n_groups=32, top_groups=1), SHAPE)])  # 4 experts a group cannot hold the top 8
def test_select_refuses_bad_configs(m, bad, status):
    cfg = ctypes.byref(_cfg(m, **bad))
    L = m.lib()
    assert L.nvfp4moe_router_select(cfg, FAKE, 1024, 4, None, FAKE, FAKE, None) == status
    assert L.nvfp4moe_router_select_backward(cfg, FAKE, 1024, 4, None, FAKE, FAKE, FAKE, 1024, None) == status


def test_select_refuses_bad_arguments(m):
    L, c = m.lib(), ctypes.byref(_cfg(m))
    odd = ctypes.c_void_p(0x10002)

    def sel(cfg=c, logits=FAKE, ld=128, T=4, bias=None, ids=FAKE, probs=FAKE):
        return L.nvfp4moe_router_select(cfg, logits, ld, T, bias, ids, probs, None)

    def bwd(cfg=c, logits=FAKE, ld=128, T=4, bias=None, ids=FAKE, dp=FAKE, out=FAKE, ldo=128):
        return L.nvfp4moe_router_select_backward(cfg, logits, ld, T, bias, ids, dp, out, ldo, None)

    assert sel(cfg=None) == bwd(cfg=None) == NULL
    assert sel(ld=127) == bwd(ld=127) == bwd(ldo=127) == SHAPE
    assert sel(T=-1) == bwd(T=-1) == sel(T=1 << 31) == bwd(T=1 << 31) == SHAPE
    assert sel(logits=None) == sel(ids=None) == sel(probs=None) == NULL
    assert bwd(logits=None) == bwd(ids=None) == bwd(dp=None) == bwd(out=None) == NULL
    assert sel(logits=odd) == sel(bias=odd) == sel(ids=odd) == sel(probs=odd) == ALIGN
    assert bwd(logits=odd) == bwd(bias=odd) == bwd(ids=odd) == bwd(dp=odd) == bwd(out=odd) == ALIGN
    assert sel(T=0, logits=None, ids=None, probs=None) == 0
    assert bwd(T=0, logits=None, ids=None, dp=None, out=None) == 0
    f = L.nvfp4moe_router_logits
    assert f(FAKE, -1, 64, FAKE, 8, FAKE, None) == f(FAKE, 1, 60, FAKE, 8, FAKE, None) == SHAPE
    assert f(FAKE, 1, 64, FAKE, 0, FAKE, None) == f(FAKE, 1, 64, FAKE, 1025, FAKE, None) == SHAPE
    assert f(None, 1, 64, FAKE, 8, FAKE, None) == f(FAKE, 1, 64, None, 8, FAKE, None) == NULL
    assert f(odd, 1, 64, FAKE, 8, FAKE, None) == ALIGN
    assert f(None, 0, 64, None, 8, None, None) == 0


def _q(m, mats=1, rows=64, cols=256, layout=1, codes=0x10000, scales=0x20000):
    return ctypes.byref(m.Mxfp4Tensor(codes, scales, mats, rows, cols, layout))


def test_mxfp4_sizes(m):
    L = m.lib()
    nc, ns = ctypes.c_size_t(), ctypes.c_size_t()
    a = ctypes.byref(nc), ctypes.byref(ns)
    assert L.nvfp4moe_mxfp4_bytes(_q(m, 3, 10, 96, 0, None, None), *a) == 0
    assert (nc.value, ns.value) == (3 * 10 * 48, 3 * 10 * 3)
    # padded to 16 rows x 128 columns (codes) and 512 columns (scales)
    assert L.nvfp4moe_mxfp4_bytes(_q(m, 3, 17, 160, 1, None, None), *a) == 0
    assert (nc.value, ns.value) == (3 * 2 * 2 * 1024, 3 * 2 * 1 * 256)
    assert L.nvfp4moe_mxfp4_bytes(_q(m), None, ctypes.byref(ns)) == NULL
    assert L.nvfp4moe_mxfp4_bytes(None, *a) == NULL
    for bad, st in ((dict(cols=48), SHAPE), (dict(cols=0), SHAPE), (dict(rows=-1), SHAPE), (dict(mats=-1), SHAPE),
                    (dict(layout=2), ARG), (dict(mats=1 << 16, rows=1 << 16), SHAPE)):
        assert L.nvfp4moe_mxfp4_bytes(_q(m, **bad), *a) == st, bad
    w = L.nvfp4moe_mxfp4_workspace_bytes
    assert w(100, 160, 4) >= 100 * (128 + 16) + 4 * 16 and w(100, 160, 4) % 256 == 0
    assert w(0, 32, 1) > 0
    assert w(-1, 32, 1) == w(4, 40, 1) == w(4, 0, 1) == w(4, 32, 0) == w(4, 32, 1025) == w(1 << 31, 32, 1) == 0
    with pytest.raises(m.Nvfp4Error):
        m.mxfp4_workspace_bytes(4, 33)


def test_mxfp4_refuses_bad_arguments(m):
    L = m.lib()
    odd = ctypes.c_void_p(0x10008)
    f, d = L.nvfp4moe_mxfp4_quantize, L.nvfp4moe_mxfp4_dequantize
    assert f(FAKE, 256, _q(m), 2, None) == ARG and f(FAKE, 256, None, 0, None) == d(None, FAKE, 256, None) == NULL
    assert f(FAKE, 248, _q(m), 0, None) == d(_q(m), FAKE, 248, None) == SHAPE
    assert f(FAKE, 260, _q(m), 0, None) == f(odd, 256, _q(m), 0, None) == d(_q(m), odd, 256, None) == ALIGN
    assert f(None, 256, _q(m), 0, None) == f(FAKE, 256, _q(m, codes=None), 0, None) == d(_q(m), None, 256, None) == NULL
    assert f(FAKE, 256, _q(m, codes=0x10008), 0, None) == f(FAKE, 256, _q(m, scales=0x10002), 0, None) == ALIGN
    assert f(None, 256, _q(m, rows=0, codes=None), 0, None) == d(_q(m, mats=0, codes=None), None, 256, None) == 0

    ws = L.nvfp4moe_mxfp4_workspace_bytes(4, 256, 1)

    def lin(x=FAKE, M=4, ldx=256, q=_q(m), out=FAKE, ldo=64, up=0, work=FAKE, n=ws):
        return L.nvfp4moe_mxfp4_linear(x, M, ldx, q, out, ldo, up, work, n, None)

    def grp(x=FAKE, R=4, ldx=256, off=FAKE, q=_q(m), out=FAKE, ldo=64, up=0, work=FAKE, n=ws):
        return L.nvfp4moe_mxfp4_grouped_linear(x, R, ldx, off, q, out, ldo, up, work, n, None)

    for g in (lin, grp):
        assert g(up=2) == ARG and g(q=None) == NULL
        assert g(q=_q(m, layout=0)) == g(q=_q(m, rows=0)) == g(q=_q(m, mats=0)) == SHAPE
        assert g(ldx=248) == g(ldo=63) == SHAPE
        assert g(n=ws - 1) == WORKSPACE and g(work=None) == NULL and g(work=odd) == ALIGN
        assert g(x=None) == g(out=None) == g(q=_q(m, codes=None)) == g(q=_q(m, scales=None)) == NULL
        assert g(x=odd) == g(ldx=260) == g(out=ctypes.c_void_p(0x10001)) == ALIGN
    assert lin(M=-1) == grp(R=-1) == lin(M=1 << 31) == SHAPE
    assert lin(q=_q(m, mats=2)) == SHAPE  # a dense product takes one matrix
    assert grp(off=None) == NULL and grp(off=ctypes.c_void_p(0x10002)) == ALIGN
    assert grp(q=_q(m, mats=1025)) == SHAPE
    assert lin(M=0, x=None, out=None) == grp(R=0, x=None, out=None, off=None) == 0


def test_mxfp4_refuses_more_tiles_than_a_launch_takes(m):
    """A workgroup of 256 threads a tile of 128 rows x 256 columns, fewer than 2^32 work-items a dispatch."""
    L = m.lib()
    for mats, N, M in ((1, 1 << 26, 64 * 128), (2, 1 << 25, 126 * 128)):  # 2^24 tiles each
        ws = L.nvfp4moe_mxfp4_workspace_bytes(M, 32, mats)
        q = _q(m, mats, N, 32)
        if mats == 1:
            assert L.nvfp4moe_mxfp4_linear(FAKE, M, 32, q, FAKE, N, 0, FAKE, ws, None) == SHAPE
        assert L.nvfp4moe_mxfp4_grouped_linear(FAKE, M, 32, FAKE, q, FAKE, N, 0, FAKE, ws, None) == SHAPE


def _table(m, *grads):
    return (m.Grad * len(grads))(*[m.Grad(*g) for g in grads])


def test_grad_plan(m):
    L = m.lib()
    size, n = ctypes.c_size_t(), ctypes.c_int64()
    a = ctypes.byref(size), ctypes.byref(n)
    # an FP32 tensor of three chunks, an empty one, a BF16 one that starts 6 bytes before a boundary and whose output
    # starts elsewhere, one whose output does not
    t = _table(m, (0x100000, 0x100000, 5000, 0), (None, None, 0, 0), (0x20000A, 0x300004, 5, 1), (0x40000A, 0x50000A, 20, 1))
    assert L.nvfp4moe_grad_plan_bytes(t, 4, *a) == 0 and n.value == 5 and size.value == 5 * 24
    buf = np.zeros(size.value // 8, np.uint64)
    p = buf.ctypes.data_as(ctypes.c_void_p)
    assert L.nvfp4moe_grad_plan(t, 4, p, size.value - 1) == WORKSPACE
    assert L.nvfp4moe_grad_plan(t, 4, None, size.value) == NULL
    assert L.nvfp4moe_grad_plan(t, 4, p, size.value) == 0
    got = [(int(r[0]), int(r[1]), int(r[2]) & 0xFFFFFFFF, int(r[2]) >> 32 & 0xFFFF, int(r[2]) >> 48 & 0xFF, int(r[2]) >> 56)
           for r in buf.reshape(5, 3)]
    at = 0x100000
    assert got == [(at, at, 2048, 0, 0, 1), (at + 8192, at + 8192, 2048, 0, 0, 1), (at + 16384, at + 16384, 5000 - 4096, 0, 0, 1),
                   (0x20000A, 0x300004, 5, 3, 1, 0), (0x40000A, 0x50000A, 20, 3, 1, 1)]
    big = _table(m, (0x100000, 0x100000, 603979776, 0))  # chunks of 32768 elements
    assert L.nvfp4moe_grad_plan_bytes(big, 1, *a) == 0 and n.value == 603979776 // 32768


def test_grad_plan_refusals(m):
    L = m.lib()
    size, n = ctypes.c_size_t(), ctypes.c_int64()
    a = ctypes.byref(size), ctypes.byref(n)
    f = L.nvfp4moe_grad_plan_bytes
    assert f(_table(m, (0x1000, 0x1000, 4, 2)), 1, *a) == ARG
    assert f(_table(m, (0x1000, 0x1000, -1, 0)), 1, *a) == f(_table(m, (0x1000, 0x1000, 4, 0)), -1, *a) == SHAPE
    assert f(_table(m, (None, 0x1000, 4, 0)), 1, *a) == f(_table(m, (0x1000, None, 4, 0)), 1, *a) == f(None, 1, *a) == NULL
    assert f(_table(m, (0x1002, 0x1000, 4, 0)), 1, *a) == f(_table(m, (0x1000, 0x1001, 4, 1)), 1, *a) == ALIGN
    assert f(None, 0, *a) == 0 and n.value == 0
    buf = np.zeros(64, np.uint64)

    def plan(*grads):
        return L.nvfp4moe_grad_plan(_table(m, *grads), len(grads), buf.ctypes.data_as(ctypes.c_void_p), buf.nbytes)

    assert plan((0x1000, 0x1000, 4, 0), (0x1010, 0x1010, 4, 0)) == 0  # neighbours
    assert plan((0x1000, 0x2000, 4, 0), (0x1000, 0x3000, 4, 0)) == 0  # one input twice, two outputs
    assert plan((0x1000, 0x1000, 4, 0), (0x1000, 0x1000, 4, 0)) == ARG  # one tensor twice, in place
    assert plan((0x1000, 0x1008, 4, 0)) == ARG  # its own output, overlapping
    assert plan((0x1000, 0x2000, 4, 0), (0x2008, 0x3000, 4, 0)) == ARG  # an output over another's input
    assert plan((0x1000, 0x2000, 4, 0), (0x4000, 0x200C, 4, 0)) == ARG  # two outputs
    assert plan((0x1000, 0x1000, 4, 0), (0x100C, 0x3000, 4, 0)) == ARG  # an input over a tensor in place
    c = L.nvfp4moe_clip_grad_norm
    ws = L.nvfp4moe_clip_workspace_bytes()
    assert c(FAKE, -1, 1.0, FAKE, FAKE, ws, None) == SHAPE
    assert c(FAKE, 1, -1.0, FAKE, FAKE, ws, None) == c(FAKE, 1, float("nan"), FAKE, FAKE, ws, None) == ARG
    assert c(None, 1, 1.0, FAKE, FAKE, ws, None) == c(FAKE, 1, 1.0, None, FAKE, ws, None) == NULL
    assert c(FAKE, 1, 1.0, FAKE, None, ws, None) == NULL and c(FAKE, 1, 1.0, FAKE, FAKE, ws - 1, None) == WORKSPACE
    assert c(FAKE, 1, 1.0, ctypes.c_void_p(0x10004), FAKE, ws, None) == ALIGN


def test_bindings_refuse_host_tensors_and_wrong_types(m):
    import torch
    l = torch.zeros(4, 16)
    for call in (lambda: m.router_select(l, 2), lambda: m.mxfp4_quantize(torch.zeros(4, 64, dtype=torch.bfloat16)),
                 lambda: m.router_select(l.half(), 2), lambda: m.router_select(l.t(), 2),
                 lambda: m.router_select(l, 2, bias=torch.zeros(15)),
                 lambda: m.router_select_backward(l, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)),
                 lambda: m.router_select_backward(l, torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)),
                 lambda: m.mxfp4_quantize(torch.zeros(4, 64)), lambda: m.GradSet([]),
                 lambda: m.GradSet([torch.zeros(4, dtype=torch.float64)]), lambda: m.GradSet([torch.zeros(4, 4)[:, :2]]),
                 lambda: m.GradSet([torch.zeros(4)], [torch.zeros(5)]), lambda: m.GradSet([torch.zeros(4)], [])):
        with pytest.raises(ValueError):
            call()


# --- the plain forms themselves ---------------------------------------------------------------------

def test_plain_select_by_hand():
    l = np.log(np.array([1.0, 2.0, 4.0, 1.0]))
    ids, p = R.select_row(l, 2)
    assert ids.tolist() == [2, 1] and np.allclose(p, [2 / 3, 1 / 3])
    ids, p = R.select_row(l, 2, renorm=False, scale=2.0)
    assert np.allclose(p, [1.0, 0.5])
    assert R.select_row(np.zeros(4), 3)[0].tolist() == [0, 1, 2]  # ties to the lower id
    ids, p = R.select_row([np.nan, 1.0, -np.inf, 0.5], 3)
    assert ids.tolist() == [1, 3, 0] and p[2] == 0.0
    ids, p = R.select_row(l, 2, bias=[10.0, 0, -np.inf, 0])
    assert ids.tolist() == [0, 1]
    # two groups: {0, 1} has the best expert, {2, 3} the better pair
    v = np.array([5.0, -9.0, 4.0, 4.0])
    assert R.select_row(v, 1, n_groups=2, top_groups=1)[0].tolist() == [0]
    assert R.select_row(v, 1, sigmoid=True, n_groups=2, top_groups=1, top2=True)[0].tolist() == [2]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_plain_gradient_against_differences(sigmoid, renorm):
    rng = np.random.default_rng(1)
    l, dp = rng.standard_normal(9) * 2, rng.standard_normal(3)
    ids, _ = R.select_row(l, 3, sigmoid=sigmoid, renorm=renorm, scale=1.5)

    def f(x):
        u, c = R.usable_logits(x)
        return 1.5 * (R.weights(c[ids], u[ids], sigmoid, renorm, R.scores(c, u, sigmoid)[ids]) * dp).sum()

    h = 1e-5
    num = np.array([(f(l + h * e) - f(l - h * e)) / (2 * h) for e in np.eye(9)])
    got = R.select_backward_row(l, ids, dp, sigmoid=sigmoid, renorm=renorm, scale=1.5)
    assert np.abs(num - got).max() < 1e-9  # h^2 |f'''| / 6 and FP64 noise 1e-16 / h


def test_plain_mxfp4_by_hand():
    bits = R.bf16_round(np.array([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] + [0.0] * 24]))
    code, byte = R.mxfp4_quantize(bits, False)
    assert byte[0, 0] == 127 and code[0, :8].tolist() == [7, 0, 2, 2, 4, 4, 6, 6]  # every tie to the even code
    seven = R.bf16_round(np.array([[7.0] + [0.0] * 31]))
    assert R.mxfp4_quantize(seven, False)[1][0, 0] == 127 and R.mxfp4_quantize(seven, True)[1][0, 0] == 128
    assert R.mxfp4_values(*R.mxfp4_quantize(seven, False))[0, 0] == 6.0  # clipped
    assert R.mxfp4_values(*R.mxfp4_quantize(seven, True))[0, 0] == 8.0
    zero = np.full((1, 32), 0x8000, np.uint16)
    code, byte = R.mxfp4_quantize(zero, True)
    assert byte[0, 0] == 0 and (code == 8).all()
