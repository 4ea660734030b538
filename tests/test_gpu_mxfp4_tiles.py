"""GPU MXFP4 products in the tile kernels (tests/test_gpu_mxfp4.py covers the few-row kernel and the quantizers): tiles of
256 columns, taken from 144 of them on, at every number of 128-column chunks modulo four and every height of a row tile;
the row-tile table that a grouped product builds on the GPU, with hostile offsets and with more experts than one wavefront
scans; a table rebuilt on the replay of a graph.

Every row is compared bit for bit with the few-row kernel (up to 8 rows of at most 2176 columns a call, within its limits
of 16 rows and 32768 elements of one matrix), and samples with FP64 under the bars of tests/test_gpu_mxfp4.py.  The
few-row kernel itself with rows that are few on average only."""
import numpy as np
import pytest

from tests import plain_ops as R
from tests.helpers import to_dev, to_host
from tests.test_gpu_mxfp4 import OFFSETS, _bits, _check_product, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_moe_expert_sort_amd as m
    m.lib()
    return m, torch.device("cuda:0")


def _by_few(m, x, w):
    """The dense product of x's rows, eight at a time."""
    import torch
    return torch.cat([m.mxfp4_linear(x[r:r + 8], w) for r in range(0, len(x), 8)])


def _sample_fp64(y, xb, wv, rows):
    xv = R.mxfp4_values(*R.mxfp4_quantize(xb[rows], False))
    _check_product(R.bf16_values(y[rows]), xv, wv)


# 1, 5, 6, 7, 9, 16 and 17 chunks of 128 columns
@pytest.mark.parametrize("K", [96, 544, 768, 864, 1056, 2048, 2176])
@pytest.mark.parametrize("last,N", [(20, 1000), (33, 1024), (64, 997), (90, 1000), (128, 776)])
def test_linear_in_wide_tiles(gpu, K, last, N):
    """36 whole row tiles and one of `last` rows by four column tiles of 256: 148 tiles."""
    import torch
    m, dev = gpu
    M = 36 * 128 + last
    assert ((M + 127) // 128) * ((N + 255) // 256) >= 144
    rng = np.random.default_rng(K + last)
    w, wv = _weights(m, dev, _bits(rng, (1, N, K), 0.05))
    xb = _bits(rng, (M, K))
    xb[:, ::7] = R.bf16_round(R.bf16_values(xb[:, ::7]) * 20)
    x = to_dev(xb, dev)
    out = torch.full((M + 2, N), 77, dtype=torch.int16, device=dev)
    m.mxfp4_linear(x, w, out=out[1:-1])
    assert (out[0] == 77).all() and (out[-1] == 77).all()
    y = out[1:-1]
    assert torch.equal(y, _by_few(m, x, w))
    _sample_fp64(to_host(y), xb, wv[0], np.concatenate([rng.integers(0, M, 12), np.arange(M - 4, M)]))


@pytest.mark.parametrize("K", [96, 544, 768, 864, 1056, 2048, 2176])
@pytest.mark.parametrize("N", [1536, 1500])
def test_grouped_in_wide_tiles(gpu, K, N):
    """Experts of every tile height (up to 32, 64, 96 and 128 rows), of one row and none, rows outside the offsets."""
    import torch
    m, dev = gpu
    counts = [20, 0, 50, 90, 128, 129, 1, 700, 0, 32, 33, 257, 96, 1000]
    E, R0 = len(counts), 3
    off = R0 + np.concatenate([[0], np.cumsum(counts)])
    rows = int(off[-1]) + 5
    assert rows > 16 * E and (rows // 128 + E) * ((N + 255) // 256) >= 144
    gen = torch.Generator(device=dev).manual_seed(K + N)
    bits = (torch.randn(E, N, K, generator=gen, device=dev) * 0.1).to(torch.bfloat16).view(torch.int16)
    x = torch.randn(rows, K, generator=gen, device=dev).to(torch.bfloat16).view(torch.int16)
    xb = to_host(x)
    w = m.Mxfp4Weights(E, N, K, dev).quantize_from(bits)
    out = torch.full((rows, N), 77, dtype=torch.int16, device=dev)
    m.mxfp4_grouped_linear(x, to_dev(off.astype(np.int32), dev), w, out=out)
    assert (out[:R0] == 77).all() and (out[off[-1]:] == 77).all()
    y = to_host(out)
    for e in np.flatnonzero(counts):
        a, b = off[e], off[e + 1]
        one = m.Mxfp4Weights(1, N, K, dev).quantize_from(bits[e:e + 1])
        assert torch.equal(out[a:b], _by_few(m, x[a:b], one)), e
        if e in (0, 6, 11):
            wv = R.mxfp4_values(*R.mxfp4_quantize(to_host(bits[e]), False))
            _sample_fp64(y, xb, wv, np.unique([a, (a + b) // 2, b - 1]))


@pytest.mark.parametrize("off", OFFSETS)
@pytest.mark.parametrize("N", [72, 4096])  # tiles of 64 columns, and of 256
def test_grouped_offsets_in_tiles(gpu, off, N):
    """Offsets of 41 rows scaled to 700: empty experts, rows outside them (left as they were), out of range and decreasing
    ones."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(13)
    rows, E, K = 700, 4, 160
    off = [o * 17 + (o % 5) for o in off]
    assert rows > 16 * E and ((rows // 128 + E) * ((N + 255) // 256) >= 144) == (N == 4096)
    bits = _bits(rng, (E, N, K), 0.1)
    w = m.Mxfp4Weights(E, N, K, dev).quantize_from(to_dev(bits, dev))
    x = to_dev(_bits(rng, (rows, K)), dev)
    out = torch.full((rows + 2, N), 77, dtype=torch.int16, device=dev)
    m.mxfp4_grouped_linear(x, torch.tensor(off, dtype=torch.int32, device=dev), w, out=out[1:-1])
    want = torch.full((rows + 2, N), 77, dtype=torch.int16, device=dev)
    o = np.maximum.accumulate(np.clip(off, 0, rows))
    for e in range(E):
        if o[e + 1] > o[e]:
            one = m.Mxfp4Weights(1, N, K, dev).quantize_from(to_dev(bits[e:e + 1], dev))
            want[1 + o[e]:1 + o[e + 1]] = _by_few(m, x[o[e]:o[e + 1]], one)
    assert torch.equal(out, want)


@pytest.mark.parametrize("off", OFFSETS)
def test_grouped_offsets_of_few_rows(gpu, off):
    """The same offsets in the few-row kernel: four more experts without rows keep the average below its limit."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(14)
    rows, E, N, K = 41, 8, 72, 160
    off = off + [off[-1], -3, 7, 1 << 30 if off[-1] > rows else off[-1]]
    assert rows <= 8 * E
    bits = _bits(rng, (E, N, K), 0.1)
    w, _ = _weights(m, dev, bits)
    x = to_dev(_bits(rng, (rows, K)), dev)
    out = torch.full((rows + 2, N), 77, dtype=torch.int16, device=dev)
    m.mxfp4_grouped_linear(x, torch.tensor(off, dtype=torch.int32, device=dev), w, out=out[1:-1])
    want = torch.full((rows + 2, N), 77, dtype=torch.int16, device=dev)
    o = np.maximum.accumulate(np.clip(off, 0, rows))
    for e in range(E):
        if o[e + 1] > o[e]:
            one, _ = _weights(m, dev, bits[e:e + 1])
            want[1 + o[e]:1 + o[e + 1]] = m.mxfp4_linear(x[o[e]:o[e + 1]], one)
    assert torch.equal(out, want)


@pytest.mark.parametrize("E,rows,N,K", [(257, 4200, 48, 64), (300, 5000, 16, 96), (777, 13001, 33, 32), (1024, 17000, 16, 64),
                                        (1024, 16385, 64, 32)])
@pytest.mark.parametrize("kind", ["skewed", "every second", "last", "first"])
def test_grouped_table_of_many_experts(gpu, E, rows, N, K, kind):
    """The table is scanned across four wavefronts, four experts a thread: skewed counts with empty experts, every second
    expert empty, all rows in the last or the first one; hostile values among the offsets of the first kind."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(E + rows)
    if kind == "skewed":
        p = np.exp(rng.standard_normal(E) * 2)
        counts = rng.multinomial(rows, p / p.sum())
    elif kind == "every second":
        p = np.where(np.arange(E) % 2 == 1, 1.0, 0.0)
        counts = rng.multinomial(rows, p / p.sum())
    else:
        counts = np.zeros(E, np.int64)
        counts[-1 if kind == "last" else 0] = rows
    off = np.concatenate([[0], np.cumsum(counts)])
    given = off.copy()
    if kind == "skewed":  # a decreasing offset counts as its predecessor, one past the rows as their end
        given[1::9] -= rng.integers(0, rows, len(given[1::9]))
        given[-1] = 1 << 30
    o = np.maximum.accumulate(np.clip(given, 0, rows))
    bits, xb = _bits(rng, (E, N, K), 0.1), _bits(rng, (rows, K))
    w, wv = _weights(m, dev, bits)
    x = to_dev(xb, dev)
    out = torch.full((rows, N), 77, dtype=torch.int16, device=dev)
    assert rows > 16 * E
    m.mxfp4_grouped_linear(x, to_dev(given.astype(np.int32), dev), w, out=out)
    y = to_host(out)
    xv = R.mxfp4_values(*R.mxfp4_quantize(xb, False))
    for e in np.flatnonzero(np.diff(o)):
        _check_product(R.bf16_values(y[o[e]:o[e + 1]]), xv[o[e]:o[e + 1]], wv[e])
    assert o[0] == 0 and o[-1] == rows  # every row belongs to an expert
    # one row of each expert that has some, through the few-row kernel: the same bits
    used = np.flatnonzero(np.diff(o))
    pick = o[used + 1] - 1
    few = np.zeros(E + 1, np.int64)
    few[used + 1] = 1
    again = m.mxfp4_grouped_linear(x[torch.from_numpy(pick).to(dev)], to_dev(np.cumsum(few).astype(np.int32), dev), w)
    assert np.array_equal(to_host(again), y[pick])


@pytest.mark.parametrize("rows", [40, 400])
def test_graphs_over_one_workspace(gpu, rows):
    """Two graphs over one workspace, replayed in turn with new rows and offsets and eager calls between: of 400 rows each
    has its quantized rows in it and one its table, of 40 the grouped product finds its passes anew."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(22)
    E, N, K = 6, 96, 256
    assert rows <= 8 * E or rows > 16 * E
    w, _ = _weights(m, dev, _bits(rng, (E, N, K), 0.1))
    one, _ = _weights(m, dev, _bits(rng, (1, N, K), 0.1))
    x = to_dev(_bits(rng, (rows, K)), dev)
    off = torch.tensor([0, 10, 10, 33, 35, 36, rows], dtype=torch.int32, device=dev)
    ws = m.mxfp4_alloc_workspace(rows, K, E, dev)
    a, b = m.mxfp4_grouped_linear(x, off, w), m.mxfp4_linear(x, one)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        m.mxfp4_grouped_linear(x, off, w, workspace=ws, out=a)
    with torch.cuda.graph(g2):
        m.mxfp4_linear(x, one, workspace=ws, out=b)
    for seed in range(4):
        r = np.random.default_rng(seed)
        x.copy_(to_dev(_bits(r, (rows, K)), dev))
        cuts = np.sort(r.integers(0, rows + 1, E - 1))
        off.copy_(torch.from_numpy(np.concatenate([[0], cuts, [rows]]).astype(np.int32)))
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        want, dense = m.mxfp4_grouped_linear(x, off, w), m.mxfp4_linear(x, one)
        assert torch.equal(a, want) and torch.equal(b, dense)
        for e, (lo, hi) in enumerate(zip(off.tolist(), off.tolist()[1:])):
            if hi > lo:  # and not the table of the replay before
                alone = torch.zeros(E + 1, dtype=torch.int32, device=dev)
                alone[e + 1:] = 1
                assert torch.equal(m.mxfp4_grouped_linear(x[hi - 1:hi], alone, w)[0], a[hi - 1])


@pytest.mark.parametrize("E,rows,N,K", [(1, 16, 40, 96), (5, 40, 72, 160), (64, 512, 33, 96), (65, 520, 80, 256),
                                        (128, 1024, 200, 320), (700, 5000, 48, 32), (1024, 8192, 16, 64)])
@pytest.mark.parametrize("kind", ["skewed", "an eighth", "last", "first", "hostile"])
def test_grouped_few_rows_on_average(gpu, E, rows, N, K, kind):
    """The few-row kernel, whose rule knows the average only: experts of many passes of 32 rows beside empty ones.  Every
    expert of more than 16 rows is compared bit for bit with its dense product in tiles, all rows with FP64."""
    import torch
    m, dev = gpu
    rng = np.random.default_rng(E * 7 + rows)
    counts = np.zeros(E, np.int64)
    if kind in ("skewed", "hostile"):
        p = np.exp(rng.standard_normal(E) * 2)
        counts = rng.multinomial(rows, p / p.sum())
    elif kind == "an eighth":
        counts = rng.multinomial(rows - rows // 8, np.full(E, 1 / E))
        counts[E // 2] += rows // 8
    else:
        counts[-1 if kind == "last" else 0] = rows
    given = np.concatenate([[0], np.cumsum(counts)])
    if kind == "hostile":
        given[1::3] -= rng.integers(0, 2 * rows, len(given[1::3]))
        given[0] = rng.integers(-5, 5)
        given[-1] += rng.integers(-3, 1 << 20)
    o = np.maximum.accumulate(np.clip(given, 0, rows))
    assert rows <= (8 if E > 1 else 16) * E and rows * K <= 32768 * E
    bits, xb = _bits(rng, (E, N, K), 0.1), _bits(rng, (rows, K))
    w, wv = _weights(m, dev, bits)
    x = to_dev(xb, dev)
    out = torch.full((rows + 2, N), 77, dtype=torch.int16, device=dev)
    m.mxfp4_grouped_linear(x, to_dev(given.astype(np.int32), dev), w, out=out[1:-1])
    y = to_host(out[1:-1])
    assert (out[0] == 77).all() and (out[-1] == 77).all() and (y[:o[0]] == 77).all() and (y[o[-1]:] == 77).all()
    xv = R.mxfp4_values(*R.mxfp4_quantize(xb, False))
    for e in np.flatnonzero(np.diff(o)):
        a, b = o[e], o[e + 1]
        _check_product(R.bf16_values(y[a:b]), xv[a:b], wv[e])
        if b - a > 16:
            one = m.Mxfp4Weights(1, N, K, dev).quantize_from(to_dev(bits[e:e + 1], dev))
            assert np.array_equal(to_host(m.mxfp4_linear(x[a:b], one)), y[a:b]), e


def test_grouped_rows_on_one_expert_cost_no_more(gpu):
    """1024 rows of 128 experts, evenly and all on one: the second call reads one expert's weights in place of all.  (With
    one workgroup row an expert it took 13 times as long as the first.)"""
    import torch
    m, dev = gpu
    E, rows, N, K = 128, 1024, 1536, 2048
    w = m.Mxfp4Weights(E, N, K, dev).quantize_from(torch.randn(E, N, K, device=dev).to(torch.bfloat16))
    x = torch.randn(rows, K, device=dev).to(torch.bfloat16)
    ws = m.mxfp4_alloc_workspace(rows, K, E, dev)
    out = torch.empty(rows, N, dtype=torch.bfloat16, device=dev)
    even = torch.arange(0, rows + 1, rows // E, dtype=torch.int32, device=dev)
    one = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    one[E // 2 + 1:] = rows

    def ms(off):
        best = float("inf")
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                m.mxfp4_grouped_linear(x, off, w, workspace=ws, out=out)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    assert ms(one) < 3 * ms(even)
