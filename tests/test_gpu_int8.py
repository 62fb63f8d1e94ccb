"""8-bit integers on the GPU against the oracle: the row quantiser and the product with a scale per token and channel.

Nothing here has a tolerance.  The quantiser's arithmetic is defined operation by operation; the product's sums are whole
numbers and exact, and the three fp32 operations behind them (conversion, product of the scales, scaling) and the rounding
to bf16 are defined as well, so results are compared bit for bit.
"""

import numpy as np
import pytest
import torch

from oracle import serving as o
from parity_util import exact

pytestmark = pytest.mark.gpu

tb = pytest.importorskip("rank_factored_linear_amd.binding")
DEV = "cuda"
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


def randn(shape, seed, sd=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * sd).to(dtype).to(DEV)


def ints(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-127, 128, shape, generator=g, dtype=I8).to(DEV)


def scales(n, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(n, generator=g) + 0.01).to(DEV)


def whole(t):
    return t.cpu().numpy().astype(np.float64)


def check_rows(q, s, x):
    want_q, want_s = o.quantize_rows_int8(exact(x))
    assert np.array_equal(whole(s), want_s, equal_nan=True)
    assert np.array_equal(whole(q), want_q)


def check_product(y, xq, xs, wq, ws):
    want = torch.from_numpy(o.row_product(whole(xq), whole(xs), whole(wq), whole(ws))).to(y.dtype)
    got = y.cpu()
    bad = (got != want) & ~(got.isnan() & want.isnan())
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


# --------------------------------------------------------------------------------------------------------------------
# Quantiser
# --------------------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n", [(1, 8), (1, 128), (3, 136), (5, 1152), (17, 2040), (6, 2056), (3, 5376), (130, 256),
                                 (2, 21504), (3, 32768), (2, 32776), (1, 65536)])
def test_rows(m, n, dtype):
    print(m, n, dtype, flush=True)
    x = randn((m, n), m + n, 3.0, dtype)
    q, s = tb.quantize_rows_int8(x)
    check_rows(q, s, x)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_row_extremes(dtype):
    """Zero rows, rows below the floor, the largest values, one bad value anywhere in a row, ties."""
    rows = []
    for top in (0.0, 1e-40, 2.0 ** -127, 1e-31, 7.9e-31, 1e-20, 126.0, 127.0, 128.0, 1e30, 3.38e38):
        rows.append((torch.linspace(-1, 1, 2056, dtype=torch.float64) * top).to(dtype))
    for at, bad in ((3, float("inf")), (2055, -float("inf")), (1024, float("nan"))):
        r = torch.ones(2056, dtype=dtype)
        r[at] = bad
        rows.append(r)
    r = torch.arange(2056, dtype=torch.float64).remainder(254).sub(126.5).to(dtype)   # k + 1/2, and 127 exactly
    r[0] = 127
    rows.append(r)
    x = torch.stack(rows).to(DEV)
    q, s = tb.quantize_rows_int8(x)
    check_rows(q, s, x)
    assert s[-4:-1].isnan().all() and (q[-4:-1] == 0).all() and s[:-4].isfinite().all()


def test_rows_write_nothing_else():
    x = randn((5, 264), 1)
    q = torch.full((7, 264), 99, dtype=I8, device=DEV)
    s = torch.full((7,), 5.0, device=DEV)
    got = tb.quantize_rows_int8(x, (q[1:6], s[1:6]))
    check_rows(*got, x)
    assert (q[[0, 6]] == 99).all() and (s[[0, 6]] == 5).all()


def test_bundle_to_int8():
    """The rebuilt weight's rows, quantised as any other."""
    s, W0 = randn((130,), 1, 0.1) + 1, randn((130, 264), 2, 0.02)
    U, V = randn((130, 24), 3, 0.05), randn((264, 24), 4, 0.05)
    q, sc = tb.reconstruct_weight_int8(s, W0, U, V)
    check_rows(q, sc, tb.reconstruct_weight(s, W0, U, V))
    q2, sc2 = tb.quantize_weight_int8(tb.reconstruct_weight(s, W0, U, V))
    assert torch.equal(q, q2) and torch.equal(sc, sc2)


# --------------------------------------------------------------------------------------------------------------------
# Product
# --------------------------------------------------------------------------------------------------------------------

SHAPES = [(1, 1, 16), (1, 16, 64), (1, 300, 48), (2, 129, 144), (3, 1536, 1152), (5, 33, 2064), (8, 256, 512), (16, 100, 272),
          (17, 260, 400), (31, 90, 1040), (33, 515, 656), (48, 64, 128), (61, 700, 1152), (64, 129, 3200), (65, 130, 272),
          (100, 257, 1168), (200, 64, 16), (256, 256, 256), (300, 515, 2064), (513, 1030, 528)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,out,n", SHAPES)
def test_product(m, out, n, dtype):
    print(m, out, n, dtype, flush=True)
    xq, wq, xs, ws = ints((m, n), 1), ints((out, n), 2), scales(m, 3), scales(out, 4)
    y = torch.full((m + 2, out), 7.0, dtype=dtype, device=DEV)
    tb.dense_forward_int8(xq, wq, ws, xs, out=y[1:-1])
    check_product(y[1:-1], xq, xs, wq, ws)
    assert (y[[0, -1]] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,out,n", SHAPES)
def test_product_quantises(m, out, n, dtype):
    """x quantised within the call: the same bits as from the quantiser first."""
    print(m, out, n, dtype, flush=True)
    x, wq, ws = randn((m, n), 1, 2.0, dtype), ints((out, n), 2), scales(out, 4)
    y = tb.dense_forward_int8(x, wq, ws)
    assert y.dtype == dtype
    check_product(y, *tb.quantize_rows_int8(x), wq, ws)


@pytest.mark.parametrize("m,out", [(1, 17), (16, 16), (64, 130), (96, 130), (600, 520)])
def test_largest_sums(m, out):
    """Every product at its largest over the longest reduction, -128 too: nothing wraps."""
    n = tb.INT8_MAX_IN_DIM
    xq, wq = torch.full((m, n), -128, dtype=I8, device=DEV), torch.full((out, n), -128, dtype=I8, device=DEV)
    wq[1::2] = 127
    one = torch.ones(max(m, out), device=DEV)
    y = tb.dense_forward_int8(xq, wq, one[:out], one[:m], out_dtype=F32)
    assert (y[:, ::2] == 2.0 ** 30).all() and (y[:, 1::2] == float(-128 * 127 * n)).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_row_is_the_same_in_any_batch(dtype):
    m, out, n = 700, 1040, 1168
    x, wq, ws = randn((m, n), 1, 1.0, dtype), ints((out, n), 2), scales(out, 4)
    y = tb.dense_forward_int8(x, wq, ws)
    for k in (1, 2, 16, 17, 40, 64, 65, 130, 300):
        assert torch.equal(tb.dense_forward_int8(x[:k], wq, ws), y[:k]), k
    assert torch.equal(tb.dense_forward_int8(x, wq[:515], ws[:515]), y[:, :515])


@pytest.mark.parametrize("m", [1, 5, 20, 70, 600])
def test_rows_without_a_scale(m):
    """A token with an infinity is NaN throughout, a zero token zero; a channel without a scale is NaN for all tokens."""
    x, wq, ws = randn((m, 272), 1), ints((600, 272), 2), scales(600, 4)
    ws[5] = float("nan")
    x[0, 7] = float("inf")
    if m > 1:
        x[1] = 0
    y = tb.dense_forward_int8(x, wq, ws)
    assert y[0].isnan().all() and y[:, 5].isnan().all()
    keep = torch.ones(600, dtype=torch.bool, device=DEV)
    keep[5] = False
    if m > 1:
        assert (y[1, keep] == 0).all()
    assert y[1:, keep].isfinite().all()


def test_no_tokens():
    wq, ws = ints((48, 64), 2), scales(48, 4)
    assert tb.dense_forward_int8(torch.empty(0, 64, dtype=BF, device=DEV), wq, ws).shape == (0, 48)
    q, s = tb.quantize_rows_int8(torch.empty(0, 64, dtype=F32, device=DEV))
    assert q.shape == (0, 64) and s.shape == (0,)
    assert tb.dense_forward_int8(q, wq, ws, s).shape == (0, 48)


def test_odd_outputs_and_unaligned_results():
    xq, xs, wq, ws = ints((70, 64), 1), scales(70, 3), ints((131, 64), 2), scales(131, 4)
    for dtype in (BF, F32):
        flat = torch.full((70 * 131 + 9,), 7.0, dtype=dtype, device=DEV)
        for k in (1, 16, 70):
            y = flat[3: 3 + k * 131].view(k, 131)
            tb.dense_forward_int8(xq[:k], wq, ws, xs[:k], out=y)
            check_product(y, xq[:k], xs[:k], wq, ws)
            assert (flat[:3] == 7).all() and (flat[3 + k * 131:] == 7).all()


@pytest.mark.parametrize("m", [1, 16, 61, 200, 777])
def test_streams_and_graphs(m):
    """Two streams at once, and a captured call replayed on new inputs: the same bits."""
    n, out = 1152, 640
    a, b = randn((m, n), 1), randn((m, n), 2)
    wq, ws = ints((out, n), 3), scales(out, 4)
    want = [tb.dense_forward_int8(x, wq, ws) for x in (a, b)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        with torch.cuda.stream(side):
            got.append(tb.dense_forward_int8(b, wq, ws))
        got.append(tb.dense_forward_int8(a, wq, ws))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[1 - i % 2]) for i, g in enumerate(got))
    x = a.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = tb.dense_forward_int8(x, wq, ws)
    for k in range(4):
        x.copy_((a, b)[k % 2])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k % 2])
        assert torch.equal(tb.dense_forward_int8(a, wq, ws), want[0])   # eager work in between


def test_two_graphs_do_not_share_a_workspace():
    m, n, out = 200, 1152, 640
    xs = [randn((m, n), k) for k in range(2)]
    wq, ws = ints((out, n), 3), scales(out, 4)
    want = [tb.dense_forward_int8(x, wq, ws) for x in xs]
    graphs, ys = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys.append(tb.dense_forward_int8(x, wq, ws))
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(3):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])


def check_on_gpu(y, xq, xs, wq, ws):
    """check_product for large results: sums below 2^53 are exact in float64, the rest as there."""
    want = (torch.mm(xq.double(), wq.double().t().contiguous()).float() * (xs[:, None] * ws[None, :])).to(y.dtype)
    bad = y != want
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


# 256 x 256 tiles: 136 whole ones with cut edges; 128 in two slices; 264 of which the last 8 are cut into eight; three
# columns, fewer than two steps of the reduction.  And 64 x 128 tiles in slices.
LARGE = [(2000, 4100, 1168), (1000, 8190, 3344), (2048, 8448, 4112), (2049, 4097, 48), (1030, 12345, 144), (777, 1152, 6912),
         (70, 5376, 21504), (130, 300, 65536)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,out,n", LARGE)
def test_large_products(m, out, n, dtype):
    print(m, out, n, dtype, flush=True)
    xq, wq, xs, ws = ints((m, n), 1), ints((out, n), 2), scales(m, 3), scales(out, 4)
    y = torch.full((m * out + 16,), 7.0, dtype=dtype, device=DEV)
    tb.dense_forward_int8(xq, wq, ws, xs, out=y[8:8 + m * out].view(m, out))
    check_on_gpu(y[8:8 + m * out].view(m, out), xq, xs, wq, ws)
    assert (y[:8] == 7).all() and (y[8 + m * out:] == 7).all()


def test_a_large_product_in_a_graph():
    m, out, n = 1000, 8190, 3344
    xs = [randn((m, n), k) for k in range(2)]
    wq, ws = ints((out, n), 2), scales(out, 4)
    want = [tb.dense_forward_int8(x, wq, ws) for x in xs]
    x, graph = xs[0].clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = tb.dense_forward_int8(x, wq, ws)
    for k in range(4):
        x.copy_(xs[k % 2])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k % 2])
        assert torch.equal(tb.dense_forward_int8(xs[1], wq, ws), want[1])


# Few tokens, many outputs: every number of 16-row tiles that a workgroup of the few-token kernel holds, cut ones too.
MANY = [(1, 24000, 144), (16, 13000, 272), (9, 11001, 80), (5, 6000, 400), (3, 40000, 64), (20, 15000, 128), (30, 10002, 256),
        (25, 6000, 272), (40, 12000, 128), (60, 7001, 160), (64, 4000, 96), (16, 3000, 4096), (2, 5000, 32768), (7, 260, 8208)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,out,n", MANY)
def test_few_tokens(m, out, n, dtype):
    print(m, out, n, dtype, flush=True)
    x, wq, ws = randn((m, n), 1, 2.0, dtype), ints((out, n), 2), scales(out, 4)
    xq, xs = tb.quantize_rows_int8(x)
    y = torch.full((m * out + 16,), 7.0, dtype=dtype, device=DEV)
    given, within = y[8:8 + m * out].view(m, out), tb.dense_forward_int8(x, wq, ws)
    tb.dense_forward_int8(xq, wq, ws, xs, out=given)
    check_on_gpu(given, xq, xs, wq, ws)
    assert torch.equal(within, given)
    assert (y[:8] == 7).all() and (y[8 + m * out:] == 7).all()
