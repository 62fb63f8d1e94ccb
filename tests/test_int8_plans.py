"""The shapes that tests run reach every kernel of the 8-bit integer product (the choice is a tunable estimate)."""

import pytest

pytest.importorskip("rank_factored_linear_amd.binding")

import int8_plans  # noqa: E402
from int8_plans import SLICED, TILES, kernel, tb  # noqa: E402
from test_gpu_int8 import MANY, SHAPES  # noqa: E402


@pytest.mark.parametrize("x_dtype", [tb.TB_INT8, tb.TB_BF16, tb.TB_F32])
@pytest.mark.parametrize("shape", TILES, ids=str)
def test_tiles(shape, x_dtype):
    assert kernel(*shape, x_dtype) == TILES[shape]


def test_slices_of_every_tile():
    assert [TILES[s][0] for s in SLICED] == ["64x64", "64x128", "128x128", "256"]
    assert all(TILES[s][-1] > 1 for s in SLICED)
    assert {k[0] for k in TILES.values() if k[-1] == 1} == {"64x64", "64x128", "128x128", "256"}


def test_every_kernel_for_few_tokens():
    """By tokens (16, 32, 64), 16-row tiles of a workgroup (five run the kernel of six) and, up to 16, where x comes from."""
    reached = set()
    for shape in SHAPES + MANY:
        for x_dtype in (tb.TB_INT8, tb.TB_BF16, tb.TB_F32):
            name, *how = kernel(*shape, x_dtype)
            if name == "few":
                tokens, rows, fused = how
                reached.add((tokens, 6 if rows == 5 else rows, x_dtype if fused else tb.TB_INT8))
    assert reached == {(1, r, x) for r in (1, 2, 3, 4, 6) for x in (tb.TB_INT8, tb.TB_BF16, tb.TB_F32)} | {
        (2, r, tb.TB_INT8) for r in (1, 2, 3, 4)} | {(4, r, tb.TB_INT8) for r in (1, 2, 3)}


def test_the_plan_counts_the_workspace():
    """The size that the plan states holds Q(x), its scales and every slice's sums."""
    for (m, out, n), how in TILES.items():
        p = int8_plans._plan(m, out, n, tb.TB_BF16, int8_plans.UNITS)
        tiles, area = (p.tile.split_tiles, 65536) if p.big else (p.tiles_m * p.tiles_n, p.tm * p.tn)
        sums = 4 * how[-1] * tiles * area if how[-1] > 1 else 0
        assert p.off_xs >= m * n and p.off_part >= p.off_xs + 4 * m and p.bytes == p.off_part + sums
