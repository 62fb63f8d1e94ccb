"""Float64 oracle of the 8-bit blocks and of the head norms with rotation.

TEST INFRASTRUCTURE ONLY, like the rest of this package: plain definitions in
NumPy that share no code with the HIP library.
"""

from __future__ import annotations

import numpy as np

BLOCK = 128


def e4m3_values() -> np.ndarray:
    """The 127 non-negative e4m3 numbers in order, by their encoding: exponent field 0 is k * 2^-9, field e >= 1 is
    (8 + k) * 2^(e - 10); the last pattern (field 15, k = 7) is NaN."""
    return np.array([(k if e == 0 else 8 + k) * 2.0 ** ((1 if e == 0 else e) - 10)
                     for e in range(16) for k in range(8) if (e, k) != (15, 7)])


def to_e4m3(v: np.ndarray) -> np.ndarray:
    """The nearest e4m3 number to each value (ties to the even pattern; NaN stays NaN).  |v| <= 448 after rounding."""
    grid = e4m3_values()
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(np.where(np.isnan(v), 0.0, v))
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    below, above = a - grid[lo], grid[hi] - a
    pick = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.isnan(v), np.nan, np.copysign(grid[pick], v))


def quantize_blocks(a: np.ndarray, rows: int, power_of_two: bool):
    """(held e4m3 values [m, n], scales [ceil(m / rows), ceil(n / 128)]) of a [m, n] float64 matrix of fp32 values in
    blocks of `rows` x 128.  fp32 scales: largest * (1 / 448) and value * (448 * (1 / largest)), each operation rounded
    to fp32."""
    m, n = a.shape
    held = np.empty((m, n))
    scales = np.empty((-(-m // rows), -(-n // BLOCK)))
    f32 = np.float32
    with np.errstate(all="ignore"):
        for i in range(scales.shape[0]):
            for j in range(scales.shape[1]):
                at = np.s_[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK]
                b = a[at]
                if not np.isfinite(b).all():
                    held[at], scales[i, j] = np.nan, np.nan
                    continue
                top = np.abs(b).max()
                if power_of_two:
                    e = -127
                    while 448.0 * 2.0 ** e < top:   # the least power of two whose 448-fold holds the block
                        e += 1
                    scales[i, j] = 2.0 ** e
                    held[at] = to_e4m3(b / scales[i, j])
                else:
                    t = f32(max(top, 2.0 ** -100))
                    scales[i, j] = f32(t * f32(f32(1) / f32(448)))
                    by = f32(f32(448) * f32(f32(1) / t))
                    held[at] = to_e4m3((b.astype(f32) * by).astype(np.float64))
    return held, scales


def spread(scales: np.ndarray, rows: int, m: int, n: int) -> np.ndarray:
    """Block scales as an [m, n] matrix."""
    return np.repeat(np.repeat(scales, rows, 0)[:m], BLOCK, 1)[:, :n]


def block_product(xq, xs, wq, ws) -> np.ndarray:
    """y = (xq . xs) (wq . ws)^T of held values and block scales."""
    x = xq * spread(xs, 1, *xq.shape)
    w = wq * spread(ws, BLOCK, *wq.shape)
    return x @ w.T


def head_norm_rotate(x, weight, positions, freqs, eps, offset=0.0, interleaved=False) -> np.ndarray:
    """Per-head norm and position rotation of x [tokens, heads, dim] in float64."""
    out = np.empty(x.shape)
    half = len(freqs)
    for t in range(x.shape[0]):
        for h in range(x.shape[1]):
            z = x[t, h] / np.sqrt(np.mean(x[t, h] ** 2) + eps)
            if weight is not None:
                z = z * (weight + offset)
            y = z.copy()
            for p in range(half):
                i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
                c, s = np.cos(positions[t] * freqs[p]), np.sin(positions[t] * freqs[p])
                y[i], y[j] = z[i] * c - z[j] * s, z[j] * c + z[i] * s
            out[t, h] = y
    return out


def quantize_rows_int8(a: np.ndarray):
    """(whole numbers [m, n], scales [m]) of a [m, n] float64 matrix of fp32 values: scale = largest * (1 / 127) and
    value * (127 * (1 / largest)), each operation rounded to fp32."""
    f32 = np.float32
    q, scales = np.zeros(a.shape), np.empty(a.shape[0])
    with np.errstate(all="ignore"):
        for t, row in enumerate(a):
            if not np.isfinite(row).all():
                scales[t] = np.nan
                continue
            top = f32(max(np.abs(row).max(), 2.0 ** -100))
            scales[t] = f32(top * f32(f32(1) / f32(127)))
            by = f32(f32(127) * f32(f32(1) / top))
            q[t] = np.rint((row.astype(f32) * by).astype(np.float64))
    return q, scales


def row_product(xq, xs, wq, ws) -> np.ndarray:
    """y = (xq wq^T) * (xs ws) of whole numbers and row scales: the sum exact (in 64-bit integers), then three fp32
    operations, as fp32 values."""
    acc = xq.astype(np.int64) @ wq.astype(np.int64).T
    with np.errstate(all="ignore"):
        return acc.astype(np.float32) * (xs.astype(np.float32)[:, None] * ws.astype(np.float32)[None, :])


def residual_norm(h, y, weight, post_norm, post_weight, gate, scale, eps, offset):
    """(h', z, a) in float64; gate [m, n] or None, spread over rows and channels."""
    def normed(x, w):
        x = x / np.sqrt(np.mean(x ** 2, axis=1, keepdims=True) + eps)
        return x if w is None else x * (w + offset)

    a = np.zeros_like(h)
    if y is not None:
        a = normed(y, post_weight) if post_norm else y
        if gate is not None:
            a = a * gate
    out = scale * h + a
    return out, normed(out, weight), a


def pair_places(axes, pairs: str):
    """[(i, j)] of each rotated pair: "half", "interleaved", or "axis" (in its axis's own span)."""
    half, got = len(axes), []
    for p, axis in enumerate(axes):
        if pairs == "half":
            got.append((p, p + half))
        elif pairs == "interleaved":
            got.append((2 * p, 2 * p + 1))
        else:
            first, count = axes.index(axis), axes.count(axis)
            got.append((2 * first + (p - first), 2 * first + (p - first) + count))
    return got


def head_norm_rotate_axes(x, weight, positions, axes, freqs, eps, offset, pairs: str, norm: bool) -> np.ndarray:
    """head_norm_rotate of tokens with positions [axes, tokens], in float64."""
    z = x / np.sqrt(np.mean(x ** 2, axis=2, keepdims=True) + eps) if norm else x.copy()
    if weight is not None:
        z = z * (weight + offset)
    y = z.copy()
    for p, (i, j) in enumerate(pair_places(list(axes), pairs)):
        angle = positions[axes[p]] * freqs[p]
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        y[:, :, i], y[:, :, j] = z[:, :, i] * c - z[:, :, j] * s, z[:, :, j] * c + z[:, :, i] * s
    return y
