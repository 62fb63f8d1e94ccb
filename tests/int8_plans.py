"""Which kernel of the 8-bit integer product a call takes, asked of the library's own plan, and shapes for every one.

A shape is (tokens, out_dim, in_dim).  The plan is a cost estimate that may be tuned; tests that mean to reach a kernel
take their shapes from here, and test_int8_plans.py fails where a shape no longer reaches it.
"""

import ctypes

from rank_factored_linear_amd import binding as tb

UNITS = 256   # compute units of an MI355X


class _Tiles(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("tiles_m", "tiles_n", "split_tiles", "S", "grid", "xcd_major")]
    _fields_ += [("part_bytes", ctypes.c_size_t)]


class _Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("decode", "fused", "rows", "big")] + [("tile", _Tiles)]
    _fields_ += [(n, ctypes.c_int) for n in ("tm", "tn", "tiles_m", "tiles_n", "S")]
    _fields_ += [(n, ctypes.c_size_t) for n in ("off_xq", "off_xs", "off_part", "bytes")]


_plan = tb.lib["_ZN2tb9plan_int8Elll8tb_dtypei"]   # tb::plan_int8 (tb_host.h)
_plan.restype = _Plan
_plan.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_int]


def kernel(m, out, n, x_dtype=tb.TB_INT8, units=UNITS):
    """("few", 16-token tiles, 16-row tiles, quantises x itself), ("256", tiles, cut ones, slices) or ("64x128", slices)."""
    p = _plan(m, out, n, x_dtype, units)
    if p.decode:
        tokens = 1 if m <= 16 else 2 if m <= 32 else 4
        return "few", tokens, (p.rows + 15) // 16, bool(p.fused)
    if p.big:
        return "256", p.tile.tiles_m * p.tile.tiles_n, p.tile.split_tiles, p.tile.S
    return f"{p.tm}x{p.tn}", p.S


# Every tile size, whole and in slices, with cut edges: {shape: kernel()}.
TILES = {
    (777, 1152, 6912): ("64x64", 1),
    (65, 129, 4112): ("64x64", 7),
    (64, 20001, 2064): ("64x128", 1),
    (200, 4100, 4112): ("64x128", 1),
    (300, 1649, 9840): ("64x128", 3),
    (70, 2050, 21504): ("64x128", 7),
    (1000, 8190, 3344): ("128x128", 1),
    (70, 5376, 21504): ("128x128", 6),
    (2000, 4100, 1168): ("256", 136, 0, 1),
    (2048, 8448, 4112): ("256", 264, 8, 8),       # the last eight tiles cut
    (1000, 5376, 21504): ("256", 84, 84, 3),      # every tile cut
    (200, 8200, 12304): ("256", 33, 33, 7),
}
SLICED = [(65, 129, 4112), (300, 1649, 9840), (70, 5376, 21504), (200, 8200, 12304)]   # one of each size
