"""GPU MXFP4 (nvfp4moe_mxfp4_*): quantizer and dequantizer bit for bit against the definition, products against FP64.

Bars for a product of length K: FP32 accumulation, |y - exact| <= 2 K 2^-24 sum |a w| and one BF16 rounding (2^-8
relative).  With all scales equal every partial sum is a multiple of the smallest product below 2^24 of them, so the
FP32 sum is exact and the result is the exact sum rounded to BF16."""
import numpy as np
import pytest

from tests import plain_ops as R
from tests.helpers import to_dev, to_host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_moe_expert_sort_amd as m
    m.lib()
    return m, torch.device("cuda:0")


def _bits(rng, shape, std=1.0):
    return R.bf16_round(rng.standard_normal(shape) * std)


def _nibbles(codes):
    c = codes.cpu().numpy()
    return np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)


def _every_pattern():
    """Rows whose blocks hold every BF16 pattern, under block maxima from the smallest to the largest."""
    rng = np.random.default_rng(0)
    p = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    p = p[(p & 0x7FFF) < 0x7F80]  # finite
    order = np.argsort(p & 0x7FFF, kind="stable")  # neighbours in magnitude share a block
    near = p[order][:len(p) // 32 * 32].reshape(-1, 32)
    mixed = rng.permutation(p)[:len(p) // 32 * 32].reshape(-1, 32)
    # each element beside a larger one in its block: every exponent distance up to 6
    e = np.maximum((near & 0x7F80).astype(int) + (rng.integers(0, 7, near.shape) << 7), 0)
    lead = np.minimum(e, 0x7F00).astype(np.uint16) | rng.integers(0, 128, near.shape).astype(np.uint16)
    led = near.copy()
    led[:, 0] = lead.max(1)
    return np.concatenate([near, mixed, led])


@pytest.mark.parametrize("up", [False, True])
def test_quantize_every_bf16_pattern(gpu, up):
    m, dev = gpu
    bits = _every_pattern()
    codes, scales = m.mxfp4_quantize(to_dev(bits, dev), 1 if up else 0)
    want, byte = R.mxfp4_quantize(bits, up)
    assert np.array_equal(scales.cpu().numpy(), byte)
    got = _nibbles(codes)
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (3, 96, 0), (5, 64, 8), (17, 2048, 0), (33, 1056, 24), (257, 160, 0)])
def test_quantize_sizes_strides_and_layouts(gpu, up, rows, cols, pad):
    import torch
    m, dev = gpu
    rng = np.random.default_rng(rows + cols)
    wide = _bits(rng, (rows, cols + pad), 3.0)
    wide[rng.random(wide.shape) < 0.05] = 0
    bits = np.ascontiguousarray(wide[:, :cols])
    bits[0, :32] = 0x8000  # a block of -0
    wide[:, :cols] = bits
    x = to_dev(wide, dev)[:, :cols]
    codes, scales = m.mxfp4_quantize(x, 1 if up else 0)
    want, byte = R.mxfp4_quantize(bits, up)
    assert np.array_equal(_nibbles(codes), want) and np.array_equal(scales.cpu().numpy(), byte)
    back = m.mxfp4_dequantize(codes, scales)
    assert np.array_equal(back.float().cpu().numpy(), R.mxfp4_values(want, byte).astype(np.float32))
    # the weights' tile layout: the same bytes at the documented places, zeros elsewhere
    mats = 2
    w = m.Mxfp4Weights(mats, rows, cols, dev)
    w.codes.fill_(255)
    w.scales.fill_(255)
    w.quantize_from(x.contiguous().repeat(mats, 1).view(mats, rows, cols), 1 if up else 0)
    cm, sm = R.mxfp4_tile_maps(rows, cols)
    for part, at, logical in ((w.codes, cm, codes), (w.scales, sm, scales)):
        planes = part.cpu().numpy().reshape(mats, -1)
        ref = np.zeros_like(planes)
        ref[:, at] = logical.cpu().numpy()
        assert np.array_equal(planes, ref)
    assert torch.equal(w.dequantize(), back.expand(mats, rows, cols))


def test_nonfinite_blocks_are_nan(gpu):
    import torch
    m, dev = gpu
    x = torch.randn(4, 96, device=dev).to(torch.bfloat16)
    x[1, 40] = torch.inf
    x[2, 95] = torch.nan
    codes, scales = m.mxfp4_quantize(x)
    assert scales[1].tolist()[1] == 255 and scales[2].tolist()[2] == 255 and int((scales == 255).sum()) == 2
    back = m.mxfp4_dequantize(codes, scales)
    nan = torch.zeros_like(back, dtype=torch.bool)
    nan[1, 32:64] = nan[2, 64:] = True
    assert torch.equal(torch.isnan(back), nan)
    for M in (4, 200):  # and products of their rows, no others
        xx = x.repeat(M // 4, 1)
        w = m.Mxfp4Weights(1, 48, 96, dev).quantize_from(torch.randn(1, 48, 96, device=dev).to(torch.bfloat16))
        y = m.mxfp4_linear(xx, w)
        bad = torch.isnan(xx.float()).any(1) | torch.isinf(xx.float()).any(1)
        assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


def test_dequantize_every_code_and_scale(gpu):
    import torch
    m, dev = gpu
    rng = np.random.default_rng(4)
    codes = np.tile(np.arange(256, dtype=np.uint8), 256).reshape(256, 256)  # 16 blocks of 32 codes a row
    byte = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    got = m.mxfp4_dequantize(to_dev(codes, dev), to_dev(byte, dev)).float().cpu().numpy().astype(np.float64)
    want = R.mxfp4_values(np.stack([codes & 15, codes >> 4], -1).reshape(256, 512), byte)
    want = np.where(np.abs(want) > 3.3895313892515355e38, np.sign(want) * np.inf, want)  # beyond BF16
    assert np.array_equal(got[:255], want[:255]) and np.isnan(got[255]).all()


def _weights(m, dev, bits, up=False):
    w = m.Mxfp4Weights(*bits.shape, dev).quantize_from(to_dev(bits, dev), 1 if up else 0)
    return w, R.mxfp4_values(*R.mxfp4_quantize(bits.reshape(-1, bits.shape[2]), up)).reshape(bits.shape)


def _check_product(y, xv, wv):
    exact, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    tol = 2 * xv.shape[1] * 2.0 ** -24 * mag + 2.0 ** -8 * np.abs(exact)
    assert (np.abs(y - exact) <= tol).all(), np.abs(y - exact).max()
    den = np.linalg.norm(exact)
    assert np.linalg.norm(y - exact) <= 2.0 ** -8 * den


MS = [1, 2, 15, 16, 17, 31, 33, 48, 64, 65, 127, 129, 300]


@pytest.mark.parametrize("N,K", [(1, 32), (16, 128), (15, 96), (64, 256), (100, 160), (257, 1056), (520, 544), (130, 2048)])
def test_linear_sizes(gpu, N, K):
    m, dev = gpu
    rng = np.random.default_rng(N + K)
    w, wv = _weights(m, dev, _bits(rng, (1, N, K), 0.05))
    bits = _bits(rng, (max(MS), K))
    bits[:, ::7] = R.bf16_round(R.bf16_values(bits[:, ::7]) * 20)
    xv = R.mxfp4_values(*R.mxfp4_quantize(bits, False))
    x = to_dev(bits, dev)
    rows = None
    for M in MS[::-1]:
        y = to_host(m.mxfp4_linear(x[:M], w))
        _check_product(R.bf16_values(y), xv[:M], wv[0])
        rows = y if rows is None else rows
        assert np.array_equal(y, rows[:M])  # every batch size, every kernel: the same bits


@pytest.mark.parametrize("K", [4064, 4096, 4128, 8192])
def test_linear_long_rows(gpu, K):
    """Rows at the few-row kernel's longest and beyond, with its largest share of LDS."""
    m, dev = gpu
    rng = np.random.default_rng(K)
    w, wv = _weights(m, dev, _bits(rng, (1, 80, K), 0.05))
    bits = _bits(rng, (40, K))
    xv = R.mxfp4_values(*R.mxfp4_quantize(bits, False))
    x = to_dev(bits, dev)
    full = to_host(m.mxfp4_linear(x, w))
    _check_product(R.bf16_values(full), xv, wv[0])
    for M in (1, 3, 7, 8, 9, 17):
        assert np.array_equal(to_host(m.mxfp4_linear(x[:M], w)), full[:M])


@pytest.mark.parametrize("M,N,K", [(5, 33, 128), (40, 64, 640), (200, 300, 1152)])
def test_linear_exact_sums(gpu, M, N, K):
    """Elements that quantize to themselves under one common scale: the sums are exact, so the bits are."""
    m, dev = gpu
    rng = np.random.default_rng(M)

    def grid(shape, scale):
        v = R.E2M1[rng.integers(0, 8, shape)] * rng.choice([-1.0, 1.0], shape)
        v[..., ::32] = 6.0  # the block's scale
        return v * scale

    a, b = grid((M, K), 2.0), grid((1, N, K), 2.0 ** -5)
    w, wv = _weights(m, dev, R.bf16_round(b))
    assert np.array_equal(wv, b)
    y = to_host(m.mxfp4_linear(to_dev(R.bf16_round(a), dev), w))
    assert np.array_equal(y, R.bf16_round(a @ b[0].T))


def test_linear_scale_rounding_and_wide_scales(gpu):
    m, dev = gpu
    rng = np.random.default_rng(7)
    spread = np.exp2(rng.integers(-20, 20, (70, 10)).astype(float)).repeat(32, 1)
    bits = R.bf16_round(rng.standard_normal((70, 320)) * spread)
    for up in (False, True):
        wb = R.bf16_round(rng.standard_normal((1, 50, 320)) * np.exp2(rng.integers(-20, 20, (50, 10)).astype(float)).repeat(32, 1))
        w, wv = _weights(m, dev, wb, up)
        xv = R.mxfp4_values(*R.mxfp4_quantize(bits, up))
        for M in (3, 70):
            y = R.bf16_values(to_host(m.mxfp4_linear(to_dev(bits[:M], dev), w, scale_round=1 if up else 0)))
            exact, mag = xv[:M] @ wv[0].T, np.abs(xv[:M]) @ np.abs(wv[0]).T
            assert (np.abs(y - exact) <= 2 * 320 * 2.0 ** -24 * mag + 2.0 ** -8 * np.abs(exact)).all()


def test_linear_strides_and_neighbours(gpu):
    import torch
    m, dev = gpu
    rng = np.random.default_rng(1)
    for M, N in ((9, 70), (150, 68), (150, 71)):
        w, _ = _weights(m, dev, _bits(rng, (1, N, 192), 0.1))
        wide = to_dev(_bits(rng, (M, 224)), dev)
        x = wide[:, 16:208]
        want = m.mxfp4_linear(x.contiguous(), w)
        assert torch.equal(m.mxfp4_linear(x, w), want)
        for c0 in (0, 3, 4):
            out = torch.full((M + 2, N + 9), 77, dtype=torch.int16, device=dev)
            m.mxfp4_linear(x, w, out=out[1:M + 1, c0:c0 + N])
            assert torch.equal(out[1:M + 1, c0:c0 + N], want)
            out[1:M + 1, c0:c0 + N] = 77
            assert (out == 77).all()


OFFSETS = [[0, 0, 0, 0, 0], [0, 5, 5, 40, 41], [3, 20, 20, 21, 38], [0, 41, 41, 41, 41], [41, 41, 41, 41, 41],
           [0, 1, 2, 3, 4], [-7, 12, 9, 30, 1000], [0, 30, 10, 35, 20], [1000, 2000, 3000, 4000, 5000],
           [-5, -4, -3, -2, -1], [0, 17, 17, 33, 41]]


@pytest.mark.parametrize("off", OFFSETS)
def test_grouped_offsets(gpu, off):
    """Empty experts, rows outside the offsets (left as they were), offsets out of range and decreasing (taken as the
    nearer end and as their predecessor); every row equal to its expert's dense product."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(13)
    Rr, E, N, K = 41, 4, 72, 160
    bits = _bits(rng, (E, N, K), 0.1)
    w, _ = _weights(m, dev, bits)
    x = to_dev(_bits(rng, (Rr, K)), dev)
    out = torch.full((Rr + 2, N), 77, dtype=torch.int16, device=dev)
    m.mxfp4_grouped_linear(x, torch.tensor(off, dtype=torch.int32, device=dev), w, out=out[1:-1])
    want = torch.full((Rr + 2, N), 77, dtype=torch.int16, device=dev)
    o = np.maximum.accumulate(np.clip(off, 0, Rr))
    for e in range(E):
        one, _ = _weights(m, dev, bits[e:e + 1])
        if o[e + 1] > o[e]:
            want[1 + o[e]:1 + o[e + 1]] = m.mxfp4_linear(x[o[e]:o[e + 1]], one)
    assert torch.equal(out, want)


@pytest.mark.parametrize("E,rows,N,K,skew", [(1, 70, 40, 96, 0.0), (3, 9, 64, 128, 0.0), (8, 700, 200, 320, 0.5),
                                             (8, 2500, 96, 256, 1.5), (128, 512, 80, 256, 0.5), (64, 300, 320, 768, 2.5), (700, 900, 33, 64, 1.0),
                                             (1024, 3000, 16, 32, 0.3), (60, 1, 48, 512, 0.0)])
def test_grouped_against_fp64(gpu, E, rows, N, K, skew):
    import torch
    m, dev = gpu
    rng = np.random.default_rng(E + rows)
    p = np.exp(rng.standard_normal(E) * skew * 2)
    counts = rng.multinomial(rows, p / p.sum())
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    bits, xb = _bits(rng, (E, N, K), 0.1), _bits(rng, (rows, K))
    w, wv = _weights(m, dev, bits)
    xv = R.mxfp4_values(*R.mxfp4_quantize(xb, False))
    y = to_host(m.mxfp4_grouped_linear(to_dev(xb, dev), to_dev(off, dev), w))
    for e in np.flatnonzero(counts):
        _check_product(R.bf16_values(y[off[e]:off[e + 1]]), xv[off[e]:off[e + 1]], wv[e])
    # a row alone, and the same row elsewhere in the batch
    e = int(np.argmax(counts))
    one = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    one[e + 1:] = 1
    r = int(off[e + 1]) - 1
    alone = to_host(m.mxfp4_grouped_linear(to_dev(xb[r:r + 1], dev), one, w))
    assert np.array_equal(alone[0], y[r])


def test_one_row_of_any_stride(gpu):
    """The row stride of a single row means nothing: one that no matrix of several rows may have is accepted."""
    import torch
    m, dev = gpu
    w = m.Mxfp4Weights(1, 40, 96, dev).quantize_from(torch.randn(1, 40, 96, device=dev).to(torch.bfloat16))
    wide = torch.randn(1, 101, device=dev).to(torch.bfloat16)
    x = wide[:, :96]
    assert x.stride() == (101, 1)
    out = torch.empty(1, 43, device=dev, dtype=torch.bfloat16)
    assert torch.equal(m.mxfp4_linear(x, w, out=out[:, :40]), m.mxfp4_linear(x.clone(), w))
    same = x.contiguous().clone()
    for a, b in zip(m.mxfp4_quantize(x), m.mxfp4_quantize(same)):
        assert torch.equal(a, b)
    codes, scales = m.mxfp4_quantize(same)
    assert torch.equal(m.mxfp4_dequantize(codes, scales, out=wide[:, :96]), m.mxfp4_dequantize(codes, scales))


def test_empty_products_and_refusals(gpu):
    import torch
    m, dev = gpu
    w = m.Mxfp4Weights(1, 40, 64, dev).quantize_from(torch.zeros(1, 40, 64, dtype=torch.bfloat16, device=dev))
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=dev)
    assert m.mxfp4_linear(x, w).shape == (0, 40)
    assert m.mxfp4_grouped_linear(x, torch.zeros(2, dtype=torch.int32, device=dev), w).shape == (0, 40)
    assert m.mxfp4_quantize(x)[0].shape == (0, 32) and m.mxfp4_dequantize(*m.mxfp4_quantize(x)).shape == (0, 64)
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device=dev)
    for call in (lambda: m.mxfp4_linear(x.float(), w), lambda: m.mxfp4_linear(x[:, :32], w),
                 lambda: m.mxfp4_linear(x, w, out=torch.zeros(3, 41, dtype=torch.bfloat16, device=dev)),
                 lambda: m.mxfp4_linear(x, w, workspace=torch.zeros(4096, device=dev)),
                 lambda: m.mxfp4_grouped_linear(x, torch.zeros(3, dtype=torch.int32, device=dev), w),
                 lambda: m.mxfp4_grouped_linear(x, torch.zeros(2, dtype=torch.int64, device=dev), w),
                 lambda: m.Mxfp4Weights(1, 40, 64, dev).quantize_from(torch.zeros(1, 41, 64, dtype=torch.bfloat16, device=dev))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(m.Nvfp4Error):
        m.mxfp4_linear(x, w, workspace=torch.zeros(16, dtype=torch.uint8, device=dev))
    with pytest.raises(m.Nvfp4Error):
        m.mxfp4_quantize(torch.zeros(4, 48, dtype=torch.bfloat16, device=dev))


def test_products_on_a_side_stream_and_in_a_graph(gpu):
    """Two graphs over one workspace, replayed in turn with eager calls between: each equals its eager result."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(21)
    E, N, K, rows = 6, 96, 256, 90
    w, _ = _weights(m, dev, _bits(rng, (E, N, K), 0.1))
    one, _ = _weights(m, dev, _bits(rng, (1, N, K), 0.1))
    x = to_dev(_bits(rng, (rows, K)), dev)
    off = torch.tensor([0, 10, 10, 33, 60, 61, 90], dtype=torch.int32, device=dev)
    ws = m.mxfp4_alloc_workspace(rows, K, E, dev)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream())
    a, b = m.mxfp4_grouped_linear(x, off, w, stream=side), m.mxfp4_linear(x, one, stream=side)
    side.synchronize()
    assert torch.equal(a, m.mxfp4_grouped_linear(x, off, w)) and torch.equal(b, m.mxfp4_linear(x, one))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        m.mxfp4_grouped_linear(x, off, w, workspace=ws, out=a)
    with torch.cuda.graph(g2):
        m.mxfp4_linear(x, one, workspace=ws, out=b)
    for seed in range(3):
        r = np.random.default_rng(seed)
        x.copy_(to_dev(_bits(r, (rows, K)), dev))
        cuts = np.sort(r.integers(0, rows + 1, E - 1))
        off.copy_(torch.from_numpy(np.concatenate([[0], cuts, [rows]]).astype(np.int32)))
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, m.mxfp4_grouped_linear(x, off, w)) and torch.equal(b, m.mxfp4_linear(x, one))
