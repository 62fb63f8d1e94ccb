"""The rotation over several axes on the GPU against the float64 oracle.

Tolerance: as for one axis (test_gpu_heads.py): (z + its mate) * (the norm's gamma(D) / 2 and 11 fp32 operations, the
turn's 2^-21 and 2^-52 of the largest angle), and one rounding.  Without the norm z is exact: the turn's three operations.
"""

import numpy as np
import pytest
import torch

from oracle import serving as o
from parity_util import exact, gamma
from test_gpu_heads import frequencies, randn

pytestmark = pytest.mark.gpu

tb = pytest.importorskip("rank_factored_linear_amd.binding")
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def check(y, x, w, pos, axes, fr, pairs, norm=True, eps=1e-6, offset=0.0):
    X, W = exact(x), None if w is None else exact(w)
    P, f = pos.cpu().numpy().astype(np.float64), fr.cpu().numpy()
    want = o.head_norm_rotate_axes(X, W, P, axes, f, eps, offset, pairs, norm)
    z = np.abs(o.head_norm_rotate_axes(X, None if W is None else np.abs(W) + abs(offset), P, (), f, eps, 0.0, pairs, norm))
    mate = np.zeros_like(z)
    for i, j in o.pair_places(list(axes), pairs):
        mate[..., i], mate[..., j] = z[..., j], z[..., i]
    turn = 2.0 ** -21 + 2.0 ** -52 * np.abs(P).max(initial=0) * f.max()
    u = 2.0 ** -8 if y.dtype == BF else 2.0 ** -23
    room = (z + mate) * ((gamma(x.shape[2]) / 2 if norm else 0) + 11 * 2.0 ** -23 + turn)
    err = np.abs(exact(y) - want) - (room * (1 + u) + u * np.abs(want))
    assert (err <= 0).all(), (float(err.max()), np.unravel_index(err.argmax(), err.shape))


def grid(axes, tokens, first=0):
    g = torch.Generator().manual_seed(5)
    return (torch.randint(0, 5000, (axes, tokens), generator=g) + first).to(DEV)


def in_turn(sizes):
    return tuple(a for _, a in sorted((i, a) for a, s in enumerate(sizes) for i in range(s)))


def spans(sizes):
    return tuple(a for a, s in enumerate(sizes) for _ in range(s))


CASES = [  # tokens, q heads, k heads, head size, pairs of each axis
    (1, 4, 1, 256, (32, 48, 48)), (3, 32, 8, 128, (16, 24, 24)), (5, 3, 2, 72, (18, 18)), (4, 2, 2, 130, (1, 30, 20, 5)),
    (7, 5, 1, 80, (8, 16)), (2, 1, 3, 64, (32,)), (3, 2, 1, 6, (1, 1, 1)), (2, 2, 1, 1024, (200, 200, 112)),
    (9, 7, 5, 48, (8, 8, 8)), (2, 1, 1, 777, (100, 51, 7)), (130, 6, 2, 96, (12, 4, 24)), (2, 1, 1, 500, (64, 128))]


@pytest.mark.parametrize("pairs", ["half", "interleaved", "axis"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,hq,hk,d,sizes", CASES)
def test_parity(t, hq, hk, d, sizes, dtype, pairs):
    print(t, hq, hk, d, sizes, dtype, pairs, flush=True)
    q, k = randn((t, hq, d), 1, 2.0, dtype), randn((t, hk, d), 2, 0.3, dtype)
    wq, wk = randn((d,), 3, 0.1, dtype), randn((d,), 4, 1.0, dtype)
    pos, fr = grid(len(sizes), t), frequencies(2 * sum(sizes))
    for axes in (spans(sizes),) if pairs == "axis" else (spans(sizes), in_turn(sizes)):
        kw = dict(axes=axes, interleaved=pairs == "interleaved", axis_halves=pairs == "axis")
        got = tb.head_norm_rotate([(q, wq), (k, wk)], pos, fr, 1e-6, 1.0, **kw)
        check(got[0], q, wq, pos, axes, fr, pairs, offset=1.0)
        check(got[1], k, wk, pos, axes, fr, pairs, offset=1.0)
        got = tb.head_norm_rotate([(q, None), (k, None)], pos, fr, norm=False, **kw)
        check(got[0], q, None, pos, axes, fr, pairs, norm=False)
        check(got[1], k, None, pos, axes, fr, pairs, norm=False)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,rot", [(256, 256), (80, 32), (130, 66), (15, 14)])
def test_one_axis_is_the_plain_rotation(d, rot, dtype, interleaved):
    """Bit for bit, and so are equal positions on all axes (text)."""
    q, w, fr = randn((9, 3, d), 1, 1.0, dtype), randn((d,), 2, 1.0, dtype), frequencies(rot)
    pos = torch.arange(131000, 131009, device=DEV)
    want, = tb.head_norm_rotate([(q, w)], pos, fr, interleaved=interleaved)
    one, = tb.head_norm_rotate([(q, w)], pos[None].contiguous(), fr, interleaved=interleaved, axes=(0,) * (rot // 2))
    three, = tb.head_norm_rotate([(q, w)], pos.expand(3, 9).contiguous(), fr, interleaved=interleaved,
                                 axes=tuple(p % 3 for p in range(rot // 2)))
    assert torch.equal(one, want) and torch.equal(three, want)


def test_elements_behind_the_pairs_and_bad_neighbours():
    """Behind the rotated pairs nothing takes on a neighbour's infinity, and without the norm they are copies."""
    x = randn((4, 3, 40), 1)
    x[1, 1, 0] = float("inf")
    pos, fr, axes = grid(2, 4), frequencies(24), (0,) * 4 + (1,) * 8
    for pairs in ("half", "interleaved", "axis"):
        y, = tb.head_norm_rotate([(x, None)], pos, fr, axes=axes, norm=False, interleaved=pairs == "interleaved",
                                 axis_halves=pairs == "axis")
        assert torch.equal(y[..., 24:], x[..., 24:])
        mate = dict(o.pair_places(list(axes), pairs))[0]
        bad = (~y.isfinite()).nonzero().tolist()
        assert bad and all(b[:2] == [1, 1] and b[2] in (0, mate) for b in bad), (pairs, bad)


def test_far_positions():
    pos = torch.tensor([[0, 131071, (1 << 30) - 1, -5], [(1 << 20) - 1, 0, 7, -(1 << 20)]], device=DEV)
    q, w, fr = randn((4, 2, 64), 1, 1.0, F32), randn((64,), 2, 1.0, F32), frequencies(64, 1e6)
    axes = spans((16, 16))
    y, = tb.head_norm_rotate([(q, w)], pos, fr, axes=axes)
    check(y, q, w, pos, axes, fr, "half")


@pytest.mark.parametrize("dim", [64, 36])
def test_packed_rows_in_place_and_a_cache(dim):
    t, hq, hk = 9, 4, 2
    rows = randn((t, hq + 2 * hk, dim), 1)
    keep = rows.clone()
    q, k = rows[:, :hq], rows[:, hq:hq + hk]
    cache = torch.full((hk, 40, dim), 3.0, dtype=BF, device=DEV)
    pos, fr, w, axes = grid(2, t), frequencies(24), randn((dim,), 2), spans((4, 8))
    qo = torch.empty(t, hq, dim, dtype=BF, device=DEV)
    kw = dict(axes=axes, axis_halves=True)
    tb.head_norm_rotate([(q, w), (k, None)], pos, fr, outs=[qo, cache[:, 20:20 + t].transpose(0, 1)], **kw)
    check(qo, q.contiguous(), w, pos, axes, fr, "axis")
    check(cache[:, 20:20 + t].transpose(0, 1), k.contiguous(), None, pos, axes, fr, "axis")
    assert (cache[:, :20] == 3).all() and (cache[:, 20 + t:] == 3).all() and torch.equal(rows, keep)
    tb.head_norm_rotate([(q, w), (k, None)], pos, fr, outs=[q, k], **kw)
    assert torch.equal(q, qo) and torch.equal(k, cache[:, 20:20 + t].transpose(0, 1))
    assert torch.equal(rows[:, hq + hk:], keep[:, hq + hk:])


def test_many_tokens_no_tokens_and_a_graph():
    t, sizes = 4100, (8, 4, 4)
    q, w, axes = randn((t, 5, 32), 1), randn((32,), 3), spans(sizes)
    pos, fr = grid(3, t), frequencies(32)
    y, = tb.head_norm_rotate([(q, w)], pos, fr, axes=axes)
    at = [0, 1, 2047, 4095, 4099]
    check(y[at], q[at], w, pos[:, at], axes, fr, "half")
    few, = tb.head_norm_rotate([(q[4000:], w)], pos[:, 4000:].contiguous(), fr, axes=axes)
    assert torch.equal(few, y[4000:])
    none, = tb.head_norm_rotate([(q[:0], w)], pos[:, :0].contiguous(), fr, axes=axes)
    assert none.shape == (0, 5, 32)
    x, graph = q.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, = tb.head_norm_rotate([(x, w)], pos, fr, axes=axes)
    for k in range(3):
        x.copy_(q if k != 1 else q.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        want, = tb.head_norm_rotate([(x, w)], pos, fr, axes=axes)
        assert torch.equal(got, want)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,sizes,pairs", [(72, (18, 18), "axis"), (130, (30, 33), "half"), (15, (3, 4), "interleaved"),
                                           (250, (60, 61), "half"), (256, (32, 48, 48), "half"), (1000, (200, 201), "axis")])
def test_a_token_is_the_same_in_any_batch(d, sizes, pairs, dtype, norm):
    """However many tokens there are, which decides how many lanes hold a head."""
    t, heads, axes = 4200, 8, spans(sizes)
    x, w, fr = randn((t, heads, d), 1, 1.0, dtype), randn((d,), 2, 0.1, dtype) if norm else None, frequencies(2 * sum(sizes))
    pos = grid(len(sizes), t)
    kw = dict(axes=axes, interleaved=pairs == "interleaved", axis_halves=pairs == "axis", norm=norm)
    y, = tb.head_norm_rotate([(x, w)], pos, fr, **kw)
    at = [0, 1, 2000, 4199]
    check(y[at], x[at], w, pos[:, at], axes, fr, pairs, norm)
    for k in (1, 3, 70, 1100):
        few, = tb.head_norm_rotate([(x[7:7 + k], w)], pos[:, 7:7 + k].contiguous(), fr, **kw)
        assert torch.equal(few, y[7:7 + k]), k
        check(few[:3], x[7:7 + min(k, 3)], w, pos[:, 7:7 + min(k, 3)], axes, fr, pairs, norm)


@pytest.mark.parametrize("pairs", ["half", "interleaved", "axis"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,sizes", [(2, (1,)), (3, (1,)), (5, (1, 1)), (6, (2, 1)), (12, (2, 4)), (20, (4, 5)), (36, (9, 9)),
                                     (66, (11, 20)), (114, (17, 13, 20)), (130, (30, 35)), (180, (20, 30, 30)), (250, (61, 62)),
                                     (258, (64, 65)), (300, (40, 60, 50)), (516, (130, 128)), (1022, (200, 111, 200))])
def test_every_layout_adds_a_head_in_one_order(d, sizes, dtype, pairs):
    """Many tokens spread a head over fewer lanes than a few do: the same bits, and the oracle's values."""
    tokens = 33000 if d <= 36 else 8200 if d < 130 else 4200   # enough of them for each head size
    axes = spans(sizes)
    x, w = randn((tokens, 8, d), 1, dtype=dtype), randn((d,), 2, 0.3, dtype=dtype)
    pos, fr = grid(len(sizes), tokens), frequencies(2 * len(axes))
    kw = dict(weight_offset=1.0, axes=axes, interleaved=pairs == "interleaved", axis_halves=pairs == "axis")
    many, = tb.head_norm_rotate([(x, w)], pos, fr, **kw)
    for first in (0, tokens - 7):
        rows = slice(first, first + 7)
        few, = tb.head_norm_rotate([(x[rows].contiguous(), w)], pos[:, rows].contiguous(), fr, **kw)
        assert torch.equal(few, many[rows])
        check(few, x[rows], w, pos[:, rows], axes, fr, pairs, offset=1.0)
