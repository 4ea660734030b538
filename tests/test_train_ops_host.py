"""The balance loss and the low-rank adapters without a GPU: refusals on the host (no launch), size functions, and the
plain forms that the GPU tests compare with, against autograd."""
import ctypes

import pytest

from tests import plain_train_ops as R

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10002)
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
    base = dict(n_experts=128, top_k=8, score=0, logits_type=0, coef=0.01)
    base.update(kw)
    return ctypes.byref(m.BalanceConfig(*base.values()))


def _loss(m, cfg, logits=FAKE, ld=1024, T=4, ids=FAKE, off=FAKE, S=2, loss=FAKE, counts=FAKE, ws=FAKE, n=1 << 30):
    return m.lib().nvfp4moe_router_balance_loss(cfg, logits, ld, T, ids, off, S, loss, counts, ws, n, None)


def _back(m, cfg, logits=FAKE, ld=1024, T=4, counts=FAKE, off=FAKE, S=2, dloss=None, add=None, ld_add=0, out=FAKE, ldo=1024):
    return m.lib().nvfp4moe_router_balance_backward(cfg, logits, ld, T, counts, off, S, dloss, add, ld_add, out, ldo, None)


@pytest.mark.parametrize("bad,status", [
    (dict(score=2), ARG), (dict(logits_type=-1), ARG), (dict(coef=float("nan")), ARG), (dict(coef=float("inf")), ARG),
    (dict(n_experts=0), SHAPE), (dict(n_experts=1025), SHAPE), (dict(top_k=0), SHAPE), (dict(top_k=33), SHAPE)])
def test_balance_refuses_bad_configs(m, bad, status):
    assert _loss(m, _cfg(m, **bad)) == _back(m, _cfg(m, **bad)) == status


def test_balance_refuses_bad_arguments(m):
    c = _cfg(m)
    assert _loss(m, None) == _back(m, None) == NULL
    for bad in (dict(ld=127), dict(T=-1), dict(T=1 << 31), dict(S=0), dict(S=65537), dict(off=None, S=2)):
        assert _loss(m, c, **bad) == _back(m, c, **bad) == SHAPE, bad
    assert _back(m, c, ldo=127) == _back(m, c, add=FAKE, ld_add=127) == SHAPE
    for bad in (dict(logits=None), dict(ids=None), dict(loss=None), dict(counts=None), dict(ws=None, T=257)):
        assert _loss(m, c, **bad) == NULL, bad
    for bad in (dict(logits=None), dict(counts=None), dict(out=None)):
        assert _back(m, c, **bad) == NULL, bad
    for bad in (dict(logits=ODD), dict(ids=ODD), dict(off=ODD), dict(loss=ODD), dict(counts=ODD), dict(ws=ODD)):
        assert _loss(m, c, **bad) == ALIGN, bad
    for bad in (dict(logits=ODD), dict(counts=ODD), dict(off=ODD), dict(dloss=ODD), dict(add=ODD, ld_add=128), dict(out=ODD)):
        assert _back(m, c, **bad) == ALIGN, bad
    assert _back(m, c, add=FAKE, ld_add=256) == ARG  # in place, another stride
    assert _back(m, c, T=0, logits=None, counts=None, out=None) == 0
    need = m.lib().nvfp4moe_balance_workspace_bytes(257, 128, 2)
    assert need % 256 == 0 and _loss(m, c, T=257, n=need - 1) == WORKSPACE
    assert (m.BALANCE_ONE_LAUNCH, m.BALANCE_ONE_LAUNCH_LOGITS, m.BALANCE_ONE_LAUNCH_SEQUENCES) == (256, 32768, 4)


def test_balance_workspace(m):
    f = m.lib().nvfp4moe_balance_workspace_bytes
    assert f(0, 1, 1) > 0
    assert f(100000, 256, 1) < f(100000, 256, 50) < f(100000, 512, 50)
    assert f(-1, 8, 1) == f(1 << 31, 8, 1) == f(4, 0, 1) == f(4, 1025, 1) == f(4, 8, 0) == f(4, 8, 65537) == 0


def _ad(m, A=0x10000, B=0x20000, scale=None, n=4, rank=16, K=64, N=72):
    return ctypes.byref(m.Adapters(A, B, scale, n, rank, K, N))


def _lin(m, ad, x=FAKE, M=4, ldx=64, ids=FAKE, base=None, ldb=72, out=FAKE, ldo=72, v=None, ws=FAKE, n=1 << 40):
    return m.lib().nvfp4moe_adapter_linear(ad, x, M, ldx, ids, base, ldb, out, ldo, v, ws, n, None)


def _grad(m, ad, x=FAKE, M=4, ldx=64, ids=FAKE, v=FAKE, dy=FAKE, ldy=72, base=None, ldb=64, dx=FAKE, ldo=64, dA=FAKE, dB=FAKE,
          ws=FAKE, n=1 << 40):
    return m.lib().nvfp4moe_adapter_backward(ad, x, M, ldx, ids, v, dy, ldy, base, ldb, dx, ldo, dA, dB, ws, n, None)


@pytest.mark.parametrize("bad", [dict(n=0), dict(n=1025), dict(rank=0), dict(rank=4), dict(rank=12), dict(rank=136),
                                 dict(K=0), dict(K=60), dict(K=1 << 24), dict(N=-8), dict(N=70), dict(N=1 << 24),
                                 dict(n=1024, rank=128, K=1 << 19, N=1 << 19)])
def test_adapters_refuse_bad_sizes(m, bad):
    ad = _ad(m, **bad)
    assert _lin(m, ad, ldx=1 << 25, ldo=1 << 25) == _grad(m, ad, ldx=1 << 25, ldy=1 << 25, ldo=1 << 25) == SHAPE
    assert m.lib().nvfp4moe_adapter_workspace_bytes(ad, 4, 0) == m.lib().nvfp4moe_adapter_workspace_bytes(ad, 4, 1) == 0


def test_adapters_refuse_bad_arguments(m):
    ad = _ad(m)
    eight = ctypes.c_void_p(0x10008)  # 8-byte aligned only
    assert _lin(m, None) == _grad(m, None) == NULL
    for bad in (dict(M=-1), dict(M=1 << 26), dict(ldx=56), dict(ldo=56)):
        assert _lin(m, ad, **bad) == _grad(m, ad, **bad) == SHAPE, bad
    assert _lin(m, ad, base=eight, ldb=64) == _grad(m, ad, ldy=64) == _grad(m, ad, base=eight, ldb=56) == SHAPE
    for bad in (dict(x=None), dict(ids=None), dict(ws=None)):
        assert _lin(m, ad, **bad) == _grad(m, ad, **bad) == NULL, bad
    assert _lin(m, ad, out=None) == NULL
    for bad in (dict(v=None), dict(dy=None), dict(dx=None), dict(dA=None), dict(dB=None)):
        assert _grad(m, ad, **bad) == NULL, bad
    for bad in (_ad(m, A=None), _ad(m, B=None)):
        assert _lin(m, bad) == _grad(m, bad) == NULL
    for bad in (_ad(m, A=0x10008), _ad(m, B=0x10008), _ad(m, scale=0x10002)):
        assert _lin(m, bad) == _grad(m, bad) == ALIGN
    for bad in (dict(x=eight), dict(ldx=68), dict(ldo=76), dict(ids=ODD), dict(base=eight), dict(ws=ODD)):
        assert _lin(m, ad, **bad) == _grad(m, ad, **bad) == ALIGN, bad
    assert _lin(m, ad, out=eight) == _lin(m, ad, v=eight) == ALIGN
    for bad in (dict(v=ODD), dict(dy=eight), dict(ldy=76), dict(dx=eight), dict(dA=eight), dict(dB=eight)):
        assert _grad(m, ad, **bad) == ALIGN, bad
    assert _lin(m, ad, base=FAKE, ldb=80) == _grad(m, ad, base=FAKE, ldb=72) == ARG  # in place, another stride
    assert _lin(m, ad, M=0, x=None, ids=None, out=None, ws=None) == 0
    for back, f in ((0, _lin), (1, _grad)):
        need = m.lib().nvfp4moe_adapter_workspace_bytes(ad, 4, back)
        assert need > 0 and need % 256 == 0 and f(m, ad, n=need - 1) == WORKSPACE


def test_adapter_workspace(m):
    f = m.lib().nvfp4moe_adapter_workspace_bytes
    assert f(_ad(m, A=None, B=None), 0, 0) > 0 and f(_ad(m), -1, 0) == f(_ad(m), 1 << 26, 1) == 0
    assert f(_ad(m), 1000, 0) < f(_ad(m), 1000, 1)
    # rows by adapter, transposed adapters, w, and at most 2 M / chunk partial sums
    assert f(_ad(m, n=8, rank=64, K=4096, N=4096), 8192, 1) > 8192 * 4 + 8 * 64 * 8192 * 2 + 8192 * 64 * 4
    with pytest.raises(m.Nvfp4Error):
        m.adapter_workspace_bytes(4, 64, 72, 20, 1)


# --- the plain forms ----------------------------------------------------------------------------------

@pytest.mark.parametrize("sigmoid", [False, True])
def test_plain_balance_against_autograd(sigmoid):
    import torch
    torch.manual_seed(0)
    T, E, k = 19, 7, 3
    l = torch.randn(T, E, dtype=torch.float64, requires_grad=True)
    ids = torch.randint(0, E, (T, k))
    off = torch.tensor([2, 5, 5, 18], dtype=torch.int32)
    p = torch.sigmoid(l) / torch.sigmoid(l).sum(1, keepdim=True) if sigmoid else torch.softmax(l, 1)
    loss = 0.0
    for a, b in ((2, 5), (5, 18)):
        f = torch.stack([(ids[a:b] == e).sum() for e in range(E)]).double() * E / (k * (b - a))
        loss = loss + (f * p[a:b].sum(0)).sum()
    loss = 0.3 * loss / 16
    (loss * 1.7).backward()
    got, counts = R.balance_loss(l.detach(), ids, 0.3, sigmoid, off)
    assert abs(got - float(loss.detach())) < 1e-14
    d, bound = R.balance_backward(l.detach(), counts, k, 0.3, sigmoid, off, 1.7)
    assert torch.allclose(d, l.grad, rtol=1e-12, atol=1e-16) and (bound < 1e-4 * d.abs().max()).all()


def test_plain_adapter_against_autograd():
    import torch
    torch.manual_seed(0)
    M, K, N, rank, n = 11, 6, 5, 2, 3
    x, A, B = (torch.randn(s, dtype=torch.float64, requires_grad=True) for s in ((M, K), (n, rank, K), (n, N, rank)))
    base, dy, scale = torch.randn(M, N), torch.randn(M, N, dtype=torch.float64), torch.rand(n)
    ids = torch.randint(-1, n, (M,))
    rows = []
    for r in range(M):
        a = int(ids[r])
        rows.append(base[r].double() if a < 0 else base[r].double() + scale[a].double() * (B[a] @ (A[a] @ x[r])))
    (torch.stack(rows) * dy).sum().backward()
    out, v, _ = R.adapter_linear(x.detach(), ids, A.detach(), B.detach(), base, scale)
    assert torch.allclose(out, torch.stack(rows).detach())
    (dx, dA, dB), _ = R.adapter_backward(x.detach(), ids, A.detach(), B.detach(), v, dy, None, scale)
    assert torch.allclose(dx, x.grad) and torch.allclose(dA, A.grad) and torch.allclose(dB, B.grad)


def test_a_workspace_is_enough_for_fewer_rows(m):
    """Whatever sizes the kernels choose for a number of rows, in steps around each of their changes."""
    rows = sorted({max(0, b + d) for b in (0, 16, 64, 128, 256, 512, 1000, 1024, 2048, 4096, 8192, 16384, 32768, 65536, 131072, 1 << 20)
                   for d in (-129, -1, 0, 1, 17, 130)})
    for n, rank, K, N in ((1, 8, 64, 64), (8, 16, 4096, 4096), (3, 32, 64, 200), (128, 16, 2048, 768), (4, 64, 4096, 4096), (1024, 128, 72, 64)):
        size = m.lib().nvfp4moe_adapter_workspace_bytes
        fwd, both = ([size(_ad(m, n=n, rank=rank, K=K, N=N), M, back) for M in rows] for back in (0, 1))
        assert fwd == sorted(fwd) and both == sorted(both) and fwd[0] > 0 and all(a <= b for a, b in zip(fwd, both))
    for E, S in ((128, 1), (128, 7), (512, 1), (64, 1000), (1024, 65536)):
        sizes = [m.lib().nvfp4moe_balance_workspace_bytes(T, E, S) for T in rows]
        assert sizes == sorted(sizes) and sizes[0] > 0
