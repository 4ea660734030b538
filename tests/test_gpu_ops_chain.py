"""The entry points beside the expert forward in the runs they are made for: a training step (router logits, selection,
expert forward and backward, the router's gradient, clipping) and a layer whose experts' products are MXFP4."""
import numpy as np
import pytest

import moe_workloads as W
from tests import plain_ops as R
from tests.helpers import to_dev, to_host

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


def _bits(rng, shape, std):
    return W.f32_to_bf16_bits((rng.standard_normal(shape) * std).astype(np.float32))


def test_training_step(gpu):
    """Each operator's output equals its plain form on its own input, and the parts fit each other: the selection is
    valid routing for the expert forward, whose dprobs the router's gradient takes, whose weight gradients are clipped
    together with the router's."""
    import torch
    m, dev = gpu
    T, H, I, E, K = 65, 256, 128, 16, 4
    rng = np.random.default_rng(3)
    x, wr = to_dev(_bits(rng, (T, H), 1.0), dev), to_dev(_bits(rng, (E, H), 0.1), dev)
    w1, w2 = to_dev(_bits(rng, (E, 2 * I, H), 0.05), dev), to_dev(_bits(rng, (E, H, I), 0.05), dev)
    dout = to_dev(_bits(rng, (T, H), 1.0), dev)
    bias = torch.from_numpy((rng.standard_normal(E) * 0.1).astype(np.float32)).to(dev)
    cfg = m.make_config(H, I, E, K, max_tokens=T)
    qw = m.QuantWeights(cfg, dev).quantize_from(w1, w2)
    ws = m.alloc_workspace(cfg, dev)

    logits = m.router_logits(x, wr)
    ids, probs = m.router_select(logits, K, bias=bias, score=m.SCORE_SIGMOID, scale=2.5, n_groups=4, top_groups=2,
                                 group_score=m.GROUP_TOP2)
    out, y1 = m.moe_expert_forward_unfused(cfg, x, ids, probs, qw, ws)
    assert m.device_error(cfg, ws) == 0  # every id in range, none twice
    dx, dprobs, dw1, dw2, _ = m.moe_expert_backward(cfg, x, w1, w2, y1, ws, dout)
    dlogits = m.router_select_backward(logits, ids, dprobs, bias=bias, score=m.SCORE_SIGMOID, scale=2.5)
    xf = to_host(x)
    dwr = (dlogits.t().contiguous() @ torch.from_numpy(W.bf16_bits_to_f32(xf)).to(dev)).contiguous()
    grads = [dw1, dw2, dwr]
    before = [g.clone() for g in grads]
    norm = m.clip_grad_norm(m.GradSet(grads), 1.0)
    torch.cuda.synchronize()

    l = logits.cpu().numpy().astype(np.float64)
    for t in range(T):
        i, p = R.select_row(l[t], K, bias=bias.cpu().numpy(), sigmoid=True, scale=2.5, n_groups=4, top_groups=2, top2=True)
        assert ids[t].tolist() == i.tolist()
        assert (np.abs(probs[t].cpu().numpy() - p) <= 1.01 * U * np.abs(p)).all()
        dp = dprobs[t].cpu().numpy().astype(np.float64)
        ref = R.select_backward_row(l[t], i, dp, bias=bias.cpu().numpy(), sigmoid=True, scale=2.5)
        assert (np.abs(dlogits[t].cpu().numpy() - ref) <= 1.01 * U * np.abs(ref) + 2.0 ** -45 * np.abs(dp).max()).all()
    total = float(torch.stack([g.double().square().sum() for g in before]).sum().sqrt())
    assert abs(float(norm) - total) <= 1e-13 * total and total > 1.0
    for b, g in zip(before, grads):
        assert torch.equal(g, (b.double() * (1.0 / float(norm))).float())


@pytest.mark.parametrize("T", [1, 3, 70])
def test_mxfp4_expert_layer(gpu, T):
    """Selection, rows sorted by expert, FC1, SwiGLU, FC2 and the weighted sum, with both products in MXFP4.  Each
    product is compared with FP64 on its own input (2 K 2^-24 sum |a w| and one BF16 rounding)."""
    import torch
    m, dev = gpu
    H, I, E, K = 192, 96, 12, 3
    rng = np.random.default_rng(T)
    xb = _bits(rng, (T, H), 1.0)
    b1, b2 = _bits(rng, (E, 2 * I, H), 0.1), _bits(rng, (E, H, I), 0.1)
    W1 = m.Mxfp4Weights(E, 2 * I, H, dev).quantize_from(to_dev(b1, dev))
    W2 = m.Mxfp4Weights(E, H, I, dev).quantize_from(to_dev(b2, dev))
    x = to_dev(xb, dev)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(dev)
    ids, probs = m.router_select(logits, K)
    expert, pair = torch.sort(ids.flatten().long(), stable=True)
    offsets = torch.searchsorted(expert, torch.arange(E + 1, device=dev)).int()
    rows = x[pair // K]
    y = m.mxfp4_grouped_linear(rows, offsets, W1)
    yv = torch.from_numpy(R.bf16_values(to_host(y)).astype(np.float32)).to(dev)
    h = (torch.nn.functional.silu(yv[:, :I]) * yv[:, I:]).to(torch.bfloat16)
    z = m.mxfp4_grouped_linear(h, offsets, W2)
    out = torch.zeros(T, H, device=dev).index_add_(0, pair // K, z.float() * probs.flatten()[pair][:, None])
    assert torch.isfinite(out).all()

    def check(got, a_bits, w_bits):
        av = R.mxfp4_values(*R.mxfp4_quantize(a_bits, False))
        wv = R.mxfp4_values(*R.mxfp4_quantize(w_bits.reshape(-1, w_bits.shape[2]), False)).reshape(w_bits.shape)
        e = expert.cpu().numpy()
        exact = np.stack([wv[e[r]] @ av[r] for r in range(len(e))])
        mag = np.stack([np.abs(wv[e[r]]) @ np.abs(av[r]) for r in range(len(e))])
        assert (np.abs(got - exact) <= 2 * av.shape[1] * U * mag + 2.0 ** -8 * np.abs(exact)).all()

    check(R.bf16_values(to_host(y)), to_host(rows), b1)
    check(R.bf16_values(to_host(z.view(torch.int16))), to_host(h.view(torch.int16)), b2)
