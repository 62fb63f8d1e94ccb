"""Every kernel of the 8-bit product, whole results bit for bit.

x and w are small whole numbers times powers of two (one per token, one per weight block), chosen so that every step is
exact: the e4m3 values, products of a group of eight columns within 2^4 of one another, and sums below 2^24 units in
the last place of fp32.  So y has one right value: the sum, rounded once.  A product that is missing, doubled or read
from the wrong row, block or scale changes it.
"""

import numpy as np
import pytest
import torch

from test_gpu_fp8 import check_product, held, operands, randn

pytestmark = pytest.mark.gpu

tb = pytest.importorskip("rank_factored_linear_amd.binding")
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
SCALES = {"f32": F32, "e8m0": tb.E8M0}


def units():
    return torch.cuda.get_device_properties(0).multi_processor_count


def spread(scale, rows, m, n):
    return scale.float().repeat_interleave(rows, 0)[:m].repeat_interleave(128, 1)[:, :n]


def whole(m, out, n, kind, seed=1):
    """(x wide, xq, xs, wq, ws, exact sum in fp32)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    kb, ob = -(-n // 128), -(-out // 128)

    def ints(*shape):
        return torch.randint(-2, 3, shape, generator=g, device=DEV).float()

    def powers(*shape):
        return torch.exp2(torch.randint(-1, 3, shape, generator=g, device=DEV).float())

    x, w, xs, ws = ints(m, n), ints(out, n), powers(m, kb), powers(ob, kb)
    want = (x * spread(xs, 1, m, n)) @ (w * spread(ws, 128, out, n)).t()
    assert float(want.abs().max()) < 2 ** 22
    dt = SCALES[kind]
    return x * spread(xs, 1, m, n), x.to(tb.E4M3), xs.to(dt), w.to(tb.E4M3), ws.to(dt), want


def same(y, want):
    want = want.to(y.dtype)
    if not torch.equal(y, want):
        bad = (y != want) | y.isnan()
        at = bad.nonzero()
        raise AssertionError(f"{int(bad.sum())} of {y.numel()} wrong, first at {at[0].tolist()}, last at {at[-1].tolist()}")


def check_all(m, out, n, kind):
    """y from x in e4m3 and in bf16 and fp32, both result types, between rows that stay as they were."""
    x, xq, xs, wq, ws, want = whole(m, out, n, kind)
    for yt in (BF, F32):
        room = torch.full((m + 4, out), 5.0, dtype=yt, device=DEV)
        same(tb.dense_forward_fp8(xq, wq, ws, x_scale=xs, out=room[2:2 + m]), want)
        assert (room[:2] == 5).all() and (room[2 + m:] == 5).all()
        if kind == "e8m0":   # powers of two: quantising x within the call is exact as well
            for xt in (BF, F32):
                y = tb.dense_forward_fp8(x.to(xt), wq, ws, out_dtype=yt)
                same(y, want)
                assert torch.equal(y, tb.dense_forward_fp8(x.to(xt), wq, ws, out_dtype=yt))


# Up to 64 tokens: 1, 2, 3, 4 and 6 tiles of 16 rows a workgroup on 256 compute units, one block of columns up to more
# than the eight waves take at once, each with its ragged last block.
@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("out", [130, 1000, 6001, 12000, 14000, 16001, 21504, 30003])
@pytest.mark.parametrize("m,n", [(1, 16), (1, 2064), (5, 400), (16, 1168), (17, 144), (32, 1168), (33, 272), (64, 1168)])
def test_few_tokens(m, n, out, kind):
    print(m, out, n, kind, flush=True)
    check_all(m, out, n, kind)


@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("m,out,n", [(65, 1, 16), (65, 129, 144), (200, 1003, 2064), (777, 1152, 1168), (1030, 1300, 272),
                                     (100, 5000, 6928)])
def test_middling_tokens(m, out, n, kind):
    print(m, out, n, kind, flush=True)
    check_all(m, out, n, kind)


# Exact sums say nothing of how real data is rounded in these variants.
@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("out", [1000, 6001, 12000, 14000, 16001, 21504])
@pytest.mark.parametrize("m,dtype", [(3, BF), (16, BF), (11, F32)])
def test_fp32_results_of_few_tokens(m, out, dtype, kind):
    print(m, out, dtype, kind, flush=True)
    x, wq, ws = operands(m, out, 1168, kind, dtype=dtype)
    xq, xs = tb.quantize_activations(x, SCALES[kind])
    y = tb.dense_forward_fp8(x, wq, ws, out_dtype=F32)
    check_product(y, xq, xs, wq, ws)
    assert torch.equal(y, tb.dense_forward_fp8(xq, wq, ws, x_scale=xs, out_dtype=F32))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("m", [1, 2, 3, 7, 8, 15, 16])
def test_x_quantised_into_lds_by_its_wave(m, kind, dtype):
    """Small weights: lanes quantise for others of their wave.  The same numbers as from x quantised beforehand."""
    x, wq, ws = operands(m, 1000, 2000, kind, dtype=dtype)   # two blocks a wave, the last one ragged
    xq, xs = tb.quantize_activations(x, SCALES[kind])
    for yt in (BF, F32):
        want = tb.dense_forward_fp8(xq, wq, ws, x_scale=xs, out_dtype=yt)
        assert torch.equal(tb.dense_forward_fp8(x, wq, ws, out_dtype=yt), want)


@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("m,out", [(1, 130), (16, 12001), (33, 700), (64, 6912), (300, 520), (2041, 4099)])
def test_outliers_that_cancel(m, out, kind):
    """One product of +-448^2 in each group of eight columns, signs alternating, beside seven of 30.  fp32 y is the sum;
    bf16 y is off by at most 7 x 2^-13 of the terms' magnitudes, which here is most of the sum itself."""
    n = 1152
    x, w = torch.ones(m, n, device=DEV), torch.full((out, n), 30.0, device=DEV)
    x[:, 0::16], x[:, 8::16], w[:, 0::8] = 448, -448, 448
    ones = lambda *shape: torch.ones(*shape, device=DEV).to(SCALES[kind])   # noqa: E731
    args = x.to(tb.E4M3), w.to(tb.E4M3), ones(-(-out // 128), 9), ones(m, 9)
    want, size = 30.0 * 7 * 144, 144 * (448.0 ** 2 + 7 * 30)
    assert (tb.dense_forward_fp8(*args, out_dtype=F32) == want).all()
    off = (tb.dense_forward_fp8(*args).float() - want).abs().max().item()
    assert off <= 7 * 2.0 ** -13 * size * (1 + 2.0 ** -8) + 2.0 ** -8 * want
    print("bf16 off by", off, flush=True)


@pytest.mark.parametrize("m,out", [(5, 1000), (50, 1000), (300, 1000)])
def test_outlier_channels(m, out):
    """Activations with eight channels a hundred times as large as the others."""
    x, wq, ws = operands(m, out, 1152, "f32")
    x[:, 7::144] *= 100
    xq, xs = tb.quantize_activations(x)
    check_product(tb.dense_forward_fp8(x, wq, ws), xq, xs, wq, ws)
    check_product(tb.dense_forward_fp8(x, wq, ws, out_dtype=F32), xq, xs, wq, ws)


# ---- the 256 x 256 tiles: bf16 results with tiles for half the compute units ----------------------------------------


def tiles(m, out):
    return -(-m // 256) * -(-out // 256)


def cut_tiles(m, out, n):
    """(tiles cut into slices, slices of each), by the rule at plan_fp8_tiles."""
    rest, kb = tiles(m, out) % units(), -(-n // 128)
    s = min(units() // rest, kb // 4, 8) if rest else 1
    return (rest, s) if s > 1 and kb - kb // s > 12 else (0, 1)


def takes_tiles(m, out):
    return m > 64 and 2 * tiles(m, out) >= units()


MANY = [  # 136 tiles on 256 units; one, two, three blocks of columns and more, ragged ones; out even, odd, not wide
    (2041, 4099, 16), (2048, 4352, 128), (2041, 4104, 144), (1800, 4099, 272), (2041, 4100, 400), (2000, 4347, 1168),
    (2041, 4099, 2064),                    # (odd numbers of blocks)
    # 264 and 300 tiles: a second round, whole and cut into slices.
    (2041, 8387, 144), (2041, 8387, 2064), (2555, 7424, 2048), (2100, 8400, 2560), (4097, 4999, 1040), (2041, 8387, 4112),
    (2040, 4090, 3600)]                    # 128 tiles, all of them cut in two


@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("m,out,n", MANY)
def test_many_tokens(m, out, n, kind):
    print(m, out, n, kind, flush=True)
    assert takes_tiles(m, out)
    check_all(m, out, n, kind)


def test_the_sizes_above_reach_whole_and_cut_tiles():
    cuts = [cut_tiles(m, out, n) for m, out, n in MANY]
    assert units() == 256 and {s for _, s in cuts} >= {1, 2, 4, 8}
    assert {tiles(m, out) > 256 for (m, out, _), c in zip(MANY, cuts) if c[1] == 1} == {True, False}


@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("m,out,n", [(2041, 4099, 400), (2041, 8387, 2064)])
def test_tiles_of_real_data(m, out, n, kind):
    """x in e4m3 (scales token by token) and quantised in the call (block by block): the same bits, twice, from a
    workspace full of NaN patterns; a token that is not finite stays alone."""
    assert takes_tiles(m, out)
    x, wq, ws = operands(m, out, n, kind)
    xq, xs = tb.quantize_activations(x, SCALES[kind])
    y = tb.dense_forward_fp8(x, wq, ws)
    rows = torch.tensor(sorted({0, 1, 63, 64, 255, 256, 1111, m - 2, m - 1}), device=DEV)
    check_product(y[rows], xq[rows], xs[rows], wq, ws)
    assert torch.equal(y, tb.dense_forward_fp8(x, wq, ws))
    for xdt, args in ((BF, (x, wq, ws)), (tb.E4M3, (xq, wq, ws, xs))):
        need = tb.dense_forward_fp8_workspace_size(m, out, n, xdt, BF, SCALES[kind])
        dirty = torch.full((max(need, 256),), 0xFF, dtype=torch.uint8, device=DEV)
        assert torch.equal(y, tb.dense_forward_fp8(*args, workspace=dirty))
    x[1111, n - 1] = float("nan")
    x[300, 5] = float("inf")
    y2 = tb.dense_forward_fp8(x, wq, ws)
    assert y2[[300, 1111]].isnan().all()
    keep = torch.ones(m, dtype=torch.bool, device=DEV)
    keep[[300, 1111]] = False
    assert torch.equal(y2[keep], y[keep])
    w = randn((out, n), 2, 0.02)           # the weight that operands() made
    w[out - 5, n - 3] = float("inf")
    y3 = tb.dense_forward_fp8(xq, *tb.quantize_weight(w, SCALES[kind]), x_scale=xs)
    block = (out - 5) // 128 * 128
    assert y3[:, block:block + 128].isnan().all() and torch.equal(y3[:, :block], y[:, :block])
    assert torch.equal(y3[:, block + 128:], y[:, block + 128:])


def test_tiles_captured_and_on_another_stream():
    m, out, n = 2041, 8387, 2064
    x, wq, ws = operands(m, out, n, "f32")
    want = tb.dense_forward_fp8(x, wq, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = tb.dense_forward_fp8(x, wq, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, want)
    graphs = []
    for _ in range(2):
        xin, y, g = x.clone(), torch.empty_like(want), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tb.dense_forward_fp8(xin, wq, ws, out=y)
        graphs.append((g, xin, y))
    for step in range(3):
        for j, (g, xin, _) in enumerate(graphs):
            xin.copy_(randn(x.shape, 100 + 2 * step + j))
            g.replay()
        for g, xin, y in graphs:
            assert torch.equal(y, tb.dense_forward_fp8(xin, wq, ws))
