"""The entry points beside the expert forward on a stream that is not the tensors' own: a caller may drop its tensors right
after the call, and their memory is not handed out again while the stream still has the call's work before it."""
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


def _calls(m, dev):
    """{name: (inputs, what makes of them a call on a stream)}"""
    import torch
    g = torch.Generator(device=dev).manual_seed(1)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev).to(dtype)

    logits, bias, x, wr = randn(4096, 128), randn(128), randn(4096, 512, dtype=torch.bfloat16), randn(128, 512, dtype=torch.bfloat16)
    ids, dp = m.router_select(logits, 8)[0], randn(4096, 8)
    codes, scales = m.mxfp4_quantize(x)
    w = randn(2, 512, 512, dtype=torch.bfloat16)
    off = torch.tensor([0, 1000, 4096], dtype=torch.int32, device=dev)

    def weights(codes, scales, mats):
        W = m.Mxfp4Weights(mats, 512, 512, dev)
        W.codes, W.scales = codes, scales
        W.Wq.codes, W.Wq.scales = codes.data_ptr(), scales.data_ptr()
        return W

    W1, W2 = m.Mxfp4Weights(1, 512, 512, dev).quantize_from(w[:1]), m.Mxfp4Weights(2, 512, 512, dev).quantize_from(w)
    ws = m.mxfp4_alloc_workspace(4096, 512, 2, dev)
    def clip(g):  # (the set is made before the call: its plan's copy makes the host wait)
        grads = m.GradSet([g])
        return lambda s: m.clip_grad_norm(grads, 1.0, stream=s)

    return {
        "router_logits": ((x, wr), lambda x, wr: lambda s: m.router_logits(x, wr, stream=s)),
        "router_select": ((logits, bias), lambda l, b: lambda s: m.router_select(l, 8, bias=b, stream=s)),
        "router_select_backward": ((logits, ids, dp), lambda l, i, d: lambda s: m.router_select_backward(l, i, d, stream=s)),
        "mxfp4_quantize": ((x,), lambda x: lambda s: m.mxfp4_quantize(x, stream=s)),
        "mxfp4_dequantize": ((codes, scales), lambda c, sc: lambda s: m.mxfp4_dequantize(c, sc, stream=s)),
        "quantize_from": ((w,), lambda w: lambda s: m.Mxfp4Weights(2, 512, 512, dev).quantize_from(w, stream=s).codes),
        "dequantize": ((W2.codes, W2.scales), lambda c, sc: lambda s: weights(c, sc, 2).dequantize(stream=s)),
        "mxfp4_linear": ((x, W1.codes, W1.scales, ws), lambda x, c, sc, ws: lambda s: m.mxfp4_linear(
            x, weights(c, sc, 1), workspace=ws, stream=s)),
        "mxfp4_grouped_linear": ((x, off, W2.codes, W2.scales), lambda x, o, c, sc: lambda s: m.mxfp4_grouped_linear(
            x, o, weights(c, sc, 2), stream=s)),
        "clip_grad_norm": ((logits,), clip),
    }


@pytest.mark.parametrize("name", ["router_logits", "router_select", "router_select_backward", "mxfp4_quantize",
                                  "mxfp4_dequantize", "quantize_from", "dequantize", "mxfp4_linear",
                                  "mxfp4_grouped_linear", "clip_grad_norm"])
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
    """The stream of a capture, named: its calls are captured, and the tensors may be dropped once the graph is."""
    import torch
    m, dev = gpu
    side = torch.cuda.Stream(dev)
    l, x = torch.randn(300, 64, device=dev), torch.randn(300, 256, device=dev).to(torch.bfloat16)
    w = m.Mxfp4Weights(1, 128, 256, dev).quantize_from(torch.randn(1, 128, 256, device=dev).to(torch.bfloat16))
    m.router_select(l, 4), m.mxfp4_linear(x, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ids, probs = m.router_select(l, 4, stream=side)
        y = m.mxfp4_linear(x, w, stream=side)
    for k in range(3):
        l.normal_()
        x.normal_()
        g.replay()
        torch.cuda.synchronize()
        a, b = m.router_select(l, 4)
        assert torch.equal(ids, a) and torch.equal(probs, b) and torch.equal(y, m.mxfp4_linear(x, w))
    del g, l, x, w, ids, probs, y
    assert float(torch.ones(1 << 20, device=dev).sum()) == 1 << 20


def test_empty_tensors_on_a_named_stream(gpu):
    import torch
    m, dev = gpu
    side = torch.cuda.Stream(dev)
    l, x = torch.empty(0, 16, device=dev), torch.empty(0, 64, dtype=torch.bfloat16, device=dev)
    ids, probs = m.router_select(l, 4, stream=side)
    assert m.router_select_backward(l, ids, probs, stream=side).shape == (0, 16)
    w = m.Mxfp4Weights(1, 40, 64, dev).quantize_from(torch.zeros(1, 40, 64, dtype=torch.bfloat16, device=dev))
    assert m.mxfp4_linear(x, w, stream=side).shape == (0, 40)
    assert m.mxfp4_dequantize(*m.mxfp4_quantize(x, stream=side), stream=side).shape == (0, 64)
    norm = m.clip_grad_norm(m.GradSet([torch.empty(0, device=dev)]), 1.0, stream=side)
    side.synchronize()
    assert float(norm) == 0.0
