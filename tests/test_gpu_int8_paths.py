"""Every tile size of the 8-bit integer product, whole and in slices of in_dim: results bit for bit, alone, in graphs and
on two streams.  Shapes and what they reach are in int8_plans.py.
"""

import pytest
import torch

from test_gpu_int8 import check_on_gpu, ints, randn, scales

pytestmark = pytest.mark.gpu

tb = pytest.importorskip("rank_factored_linear_amd.binding")

from int8_plans import SLICED, TILES, kernel  # noqa: E402

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,out,n", TILES)
def test_tiles(m, out, n, dtype):
    print(m, out, n, dtype, flush=True)
    units = torch.cuda.get_device_properties(0).multi_processor_count
    if units == 256:
        assert kernel(m, out, n) == TILES[m, out, n]
    xq, wq, xs, ws = ints((m, n), 1), ints((out, n), 2), scales(m, 3), scales(out, 4)
    y = torch.full((m * out + 16,), 7.0, dtype=dtype, device=DEV)
    nbytes = tb.dense_forward_int8_workspace_size(m, out, n, torch.int8, dtype)
    # A workspace of the stated size between two guards, full of what slices must not add up.
    work = torch.full((nbytes + 512,), 0x5b, dtype=torch.uint8, device=DEV)
    tb.dense_forward_int8(xq, wq, ws, xs, out=y[8:8 + m * out].view(m, out), workspace=work[256:256 + nbytes])
    check_on_gpu(y[8:8 + m * out].view(m, out), xq, xs, wq, ws)
    assert (y[:8] == 7).all() and (y[8 + m * out:] == 7).all()
    assert (work[:256] == 0x5b).all() and (work[256 + nbytes:] == 0x5b).all()


@pytest.mark.parametrize("m,out,n", SLICED)
def test_slices_in_graphs(m, out, n):
    """Two captured calls, replayed one after the other and at once on two streams, with eager calls in between."""
    print(m, out, n, flush=True)
    data = [randn((m, n), k) for k in range(3)]
    wq, ws = ints((out, n), 2), scales(out, 4)
    want = [tb.dense_forward_int8(x, wq, ws) for x in data]
    for x, y in zip(data, want):
        xq, xs = tb.quantize_rows_int8(x)
        check_on_gpu(y, xq, xs, wq, ws)
    xs, ys, graphs = [data[0].clone(), data[1].clone()], [], []
    for x in xs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            ys.append(tb.dense_forward_int8(x, wq, ws))
    side = torch.cuda.Stream()
    for k in range(4):
        for j in range(2):
            xs[j].copy_(data[(k + j) % 3])
            ys[j].zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        eager = tb.dense_forward_int8(data[2], wq, ws)
        torch.cuda.synchronize()
        assert torch.equal(eager, want[2])
        for j in range(2):
            assert torch.equal(ys[j], want[(k + j) % 3]), (k, j)


@pytest.mark.parametrize("m,out,n", SLICED)
def test_slices_on_two_streams(m, out, n):
    print(m, out, n, flush=True)
    a, b = randn((m, n), 1), randn((m, n), 2)
    wq, ws = ints((out, n), 3), scales(out, 4)
    want = [tb.dense_forward_int8(x, wq, ws) for x in (a, b)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        with torch.cuda.stream(side):
            got.append(tb.dense_forward_int8(b, wq, ws))
        got.append(tb.dense_forward_int8(a, wq, ws))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[1 - i % 2]) for i, y in enumerate(got))


@pytest.mark.parametrize("m,out,n", [(300, 1649, 9840), (200, 8200, 12304)])
def test_a_row_is_the_same_whatever_the_slices(m, out, n):
    """The same tokens in batches that other tiles and other numbers of slices take."""
    x, wq, ws = randn((m, n), 1), ints((out, n), 2), scales(out, 4)
    y = tb.dense_forward_int8(x, wq, ws)
    for k in (1, 16, 33, 65, 100, 150):
        assert torch.equal(tb.dense_forward_int8(x[:k], wq, ws), y[:k]), k
    assert torch.equal(tb.dense_forward_int8(x, wq[:129], ws[:129]), y[:, :129])
