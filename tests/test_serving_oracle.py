"""Pins of the 8-bit and head-norm oracle: closed forms, torch's e4m3 casts and orthogonality."""

import numpy as np
import torch

from oracle import serving as o


def test_e4m3_grid_is_torchs():
    patterns = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(patterns, o.e4m3_values())


def test_rounding_agrees_with_torchs_cast():
    g = np.random.default_rng(1)
    v = np.concatenate([g.uniform(-448, 448, 20000), g.uniform(-0.02, 0.02, 20000)]).astype(np.float32)
    grid = o.e4m3_values().astype(np.float32)
    v = np.concatenate([v, (grid[1:] + grid[:-1]) / 2, -(grid[1:] + grid[:-1]) / 2])   # every tie
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o.to_e4m3(v.astype(np.float64)), want)


def test_power_of_two_scale_holds_the_block_and_no_smaller_one_does():
    for top in (448.0, np.nextafter(np.float32(448), np.float32(500)), 447.0, 1.0, 1.75, 1e-30, 3e38, 0.0):
        a = np.zeros((1, 128))
        a[0, 5] = top
        q, s = o.quantize_blocks(a, 1, True)
        assert s[0, 0] == 2.0 ** round(np.log2(s[0, 0]))
        assert 448 * s[0, 0] >= top
        assert s[0, 0] == 2.0 ** -127 or 448 * s[0, 0] / 2 < top


def test_rounding_is_off_by_half_a_step():
    g = np.random.default_rng(2)
    a = g.standard_normal((40, 300)).astype(np.float32).astype(np.float64)
    for rows in (1, 128):
        for p2 in (True, False):
            q, s = o.quantize_blocks(a, rows, p2)
            sp = o.spread(s, rows, *a.shape)
            assert (np.abs(q * sp - a) <= np.maximum(2.0 ** -4 * np.abs(a), 2.0 ** -10 * sp) * (1 + 2.0 ** -20)).all()


def test_rotation_keeps_norms_and_relative_positions():
    g = np.random.default_rng(3)
    x = g.standard_normal((2, 1, 16))
    f = 10.0 ** -np.arange(8)
    for inter in (False, True):
        dot = []
        for shift in (0, 12345):
            y = o.head_norm_rotate(x, None, np.array([3 + shift, 10 + shift]), f, 0.0, interleaved=inter)
            assert np.allclose((y ** 2).sum(2), 16)
            dot.append((y[0, 0] * y[1, 0]).sum())
        assert abs(dot[0] - dot[1]) < 1e-9
