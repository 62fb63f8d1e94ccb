"""Head norms with the position rotation on the GPU against the float64 oracle, and the path that ends in them.

Tolerance.  z is an fp32 chain: the square sum of D elements (gamma(D), halved by the root), root, reciprocal, two
products and the weight's sum (8 roundings, 2^-23 each).  The rotation adds two products and a sum (3), and its cosine
and sine are off by the turn's rounding (half a turn at most, 2^-24 of it: 1.9e-7 rad), two units in the last place
(2.4e-7) and the fp64 angle (2^-52 of position * freq): 2^-21 + that.  All of it of |z_i| + |z_j|.  y is rounded once
(bf16: 2^-8 of the value; fp32: 2^-23).
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import serving as o
from parity_util import check_forward, exact, gamma

pytestmark = pytest.mark.gpu

tb = pytest.importorskip("rank_factored_linear_amd.binding")
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def randn(shape, seed, sd=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * sd).to(dtype).to(DEV)


def frequencies(rot, base=1e4):
    half = rot // 2
    return (base ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).to(DEV)


def check(y, x, w, pos, fr, eps, offset=0.0, interleaved=False):
    X = exact(x)
    W = None if w is None else exact(w)
    p = np.zeros(x.shape[0]) if pos is None else pos.cpu().numpy().astype(np.float64)
    f = np.zeros(0) if fr is None else fr.cpu().numpy()
    want = o.head_norm_rotate(X, W, p, f, eps, offset, interleaved)
    z = np.abs(o.head_norm_rotate(X, None if W is None else np.abs(W) + abs(offset), p, f[:0], eps))
    half, D = len(f), x.shape[2]
    mate = z.copy()
    if interleaved:
        mate[..., 0:2 * half:2], mate[..., 1:2 * half:2] = z[..., 1:2 * half:2], z[..., 0:2 * half:2]
    else:
        mate[..., :half], mate[..., half:2 * half] = z[..., half:2 * half], z[..., :half]
    mate[..., 2 * half:] = 0
    turn = 2.0 ** -21 + (2.0 ** -52 * np.abs(p).max() * f.max() if half and len(p) else 0)
    u = 2.0 ** -8 if y.dtype == BF else 2.0 ** -23
    room = (z + mate) * (gamma(D) / 2 + 11 * 2.0 ** -23 + turn)
    err = np.abs(exact(y) - want) - (room * (1 + u) + u * np.abs(want))
    assert (err <= 0).all(), (float(err.max()), np.unravel_index(err.argmax(), err.shape))


CASES = [  # tokens, q heads, k heads, head size, rotated
    (1, 4, 1, 256, 256), (1, 1, 1, 2, 2), (3, 32, 8, 256, 256), (7, 5, 1, 80, 32), (2, 3, 2, 64, 64), (5, 8, 1, 128, 64),
    (4, 2, 2, 130, 66), (2, 1, 3, 96, 0), (3, 2, 1, 1, 0), (6, 3, 1, 254, 2), (2, 2, 1, 1024, 1024), (2, 1, 1, 1000, 500),
    (3, 1, 1, 15, 14), (9, 7, 5, 72, 72), (2, 2, 2, 512, 128), (130, 6, 2, 48, 16), (2, 1, 1, 777, 300)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,hq,hk,d,rot", CASES)
def test_parity(t, hq, hk, d, rot, dtype, interleaved):
    print(t, hq, hk, d, rot, dtype, interleaved, flush=True)
    q, k = randn((t, hq, d), 1, 2.0, dtype), randn((t, hk, d), 2, 0.3, dtype)
    wq, wk = randn((d,), 3, 0.1, dtype), randn((d,), 4, 1.0, dtype)
    pos = torch.arange(17, 17 + t, device=DEV)
    fr = frequencies(rot)
    for offset in (0.0, 1.0):
        got = tb.head_norm_rotate([(q, wq), (k, wk)], pos, fr, 1e-6, offset, interleaved)
        check(got[0], q, wq, pos, fr, 1e-6, offset, interleaved)
        check(got[1], k, wk, pos, fr, 1e-6, offset, interleaved)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_far_negative_and_repeated_positions(dtype):
    pos = torch.tensor([0, 131071, (1 << 20) - 1, (1 << 30) - 1, -5, 131071, -(1 << 20)], device=DEV)
    q, w = randn((len(pos), 2, 64), 1, 1.0, dtype), randn((64,), 2, 1.0, dtype)
    q[5] = q[1]
    for base in (1e4, 1e6):
        fr = frequencies(64, base)
        y, = tb.head_norm_rotate([(q, w)], pos, fr)
        check(y, q, w, pos, fr, 1e-6)
        assert torch.equal(y[1], y[5])


def test_many_tokens_take_whole_rows():
    """Enough tokens that a wave walks all heads of one."""
    t = 4100
    q, k, w = randn((t, 5, 32), 1), randn((t, 1, 32), 2), randn((32,), 3)
    pos, fr = torch.arange(t, device=DEV), frequencies(32)
    got = tb.head_norm_rotate([(q, w), (k, w)], pos, fr)
    at = [0, 1, 2047, 4095, 4096, 4099]
    check(got[0][at], q[at], w, pos[at], fr, 1e-6)
    check(got[1][at], k[at], w, pos[at], fr, 1e-6)
    few = tb.head_norm_rotate([(q[4000:], w), (k[4000:], w)], pos[4000:], fr)
    assert torch.equal(few[0], got[0][4000:]) and torch.equal(few[1], got[1][4000:])


@pytest.mark.parametrize("dim", [64, 36])
def test_packed_rows_and_a_cache(dim):
    """Views of packed q, k, v rows in, keys into the middle of a cache out; everything else stays as it was."""
    t, hq, hk = 9, 4, 2
    rows = randn((t, hq + 2 * hk, dim), 1)
    keep = rows.clone()
    q, k = rows[:, :hq], rows[:, hq:hq + hk]
    cache = torch.full((hk, 40, dim), 3.0, dtype=BF, device=DEV)   # head-major
    pos, fr, w = torch.arange(100, 100 + t, device=DEV), frequencies(dim), randn((dim,), 2)
    qo = torch.empty(t, hq, dim, dtype=BF, device=DEV)
    tb.head_norm_rotate([(q, w), (k, None)], pos, fr, outs=[qo, cache[:, 20:20 + t].transpose(0, 1)])
    check(qo, q.contiguous(), w, pos, fr, 1e-6)
    check(cache[:, 20:20 + t].transpose(0, 1), k.contiguous(), None, pos, fr, 1e-6)
    assert (cache[:, :20] == 3).all() and (cache[:, 20 + t:] == 3).all() and torch.equal(rows, keep)
    # In place on the packed rows: values and nothing else keep theirs.
    tb.head_norm_rotate([(q, w), (k, None)], pos, fr, outs=[q, k])
    assert torch.equal(q, qo) and torch.equal(k, cache[:, 20:20 + t].transpose(0, 1))
    assert torch.equal(rows[:, hq + hk:], keep[:, hq + hk:])


def test_odd_addresses_and_strides():
    big = randn((5, 3, 70), 1)
    x = big[:, :, 3:67]                       # not 16-byte aligned
    w, pos, fr = randn((64,), 2), torch.arange(5, device=DEV), frequencies(64)
    y, = tb.head_norm_rotate([(x, w)], pos, fr)
    check(y, x.contiguous(), w, pos, fr, 1e-6)
    assert torch.equal(y, tb.head_norm_rotate([(x.contiguous(), w)], pos, fr)[0])
    one = x[:1, :1].expand(5, 3, 64)          # a broadcast input
    y, = tb.head_norm_rotate([(one, w)], pos, fr)
    check(y, one.contiguous(), w, pos, fr, 1e-6)


def test_empty_and_single():
    w, fr = randn((64,), 2), frequencies(64)
    y, = tb.head_norm_rotate([(torch.empty(0, 4, 64, dtype=BF, device=DEV), w)], torch.empty(0, dtype=torch.int64, device=DEV), fr)
    assert y.shape == (0, 4, 64)
    x, none = randn((2, 3, 64), 1), torch.empty(2, 0, 64, dtype=BF, device=DEV)
    pos = torch.arange(2, device=DEV)
    got = tb.head_norm_rotate([(none, w), (x, w), (none, None)], pos, fr)
    check(got[1], x, w, pos, fr, 1e-6)
    got, = tb.head_norm_rotate([(x, w)], None, None)     # the norm alone
    check(got, x, w, None, None, 1e-6)


def test_zeros_and_non_finite_stay_in_their_head():
    x = randn((3, 4, 64), 1)
    w, pos, fr = randn((64,), 2), torch.arange(3, device=DEV), frequencies(64)
    want, = tb.head_norm_rotate([(x, w)], pos, fr)
    x[1, 2] = 0
    x[2, 1, 5] = float("nan")
    x[0, 0, 5] = float("inf")
    y, = tb.head_norm_rotate([(x, w)], pos, fr)
    assert (y[1, 2] == 0).all() and y[2, 1].isnan().all()
    same = torch.ones(3, 4, dtype=torch.bool)
    same[1, 2] = same[2, 1] = same[0, 0] = False
    assert torch.equal(y[same], want[same])


def test_captured_and_on_another_stream():
    x, w, pos, fr = randn((6, 4, 128), 1), randn((128,), 2), torch.arange(6, device=DEV), frequencies(128)
    want, = tb.head_norm_rotate([(x, w)], pos, fr)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, = tb.head_norm_rotate([(x, w)], pos, fr)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    out, g = torch.empty_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tb.head_norm_rotate([(x, w)], pos, fr, outs=[out])
    for step in range(4):
        pos += 1
        x.copy_(randn(x.shape, step))
        g.replay()
        assert torch.equal(out, tb.head_norm_rotate([(x, w)], pos, fr)[0])


# --------------------------------------------------------------------------------------------------------------------
# The path: projections, head norms, rotation
# --------------------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("m", [1, 9, 80])
def test_qkv_of_bundles(m):
    I, D, R = 1152, 128, 16
    x = randn((m, I), 1)
    fam = {n: ((1 + 0.1 * randn((rows,), 2, 1.0, F32)).to(BF), randn((rows, I), 3 + j, 0.02), randn((rows, R), 6 + j, 0.01),
               randn((I, R), 9 + j, 0.01)) for j, (n, rows) in enumerate((("q", 512), ("k", 256), ("v", 256)))}
    wq, wk = randn((D,), 20, 0.1), randn((D,), 21, 0.1)
    pos, fr = torch.arange(5, 5 + m, device=DEV), frequencies(D)
    q, k, v = tb.qkv_forward(x, fam["q"], fam["k"], fam["v"], D, pos, fr, wq, wk, weight_offset=1.0)
    assert q.shape == (m, 4, D) and k.shape == (m, 2, D) and v.shape == (m, 2, D)
    raw = tb.linear_forward_group([(x, *fam[n]) for n in "qkv"])
    check(q, raw[0].view(m, 4, D), wq, pos, fr, 1e-6, 1.0)
    check(k, raw[1].view(m, 2, D), wk, pos, fr, 1e-6, 1.0)
    assert torch.equal(v, raw[2].view(m, 2, D))
    s, W0, U, V = (exact(t) for t in fam["v"])
    check_forward(exact(v.reshape(m, -1)), exact(x), s, W0, U, V, bf16=True, what="v")


@pytest.mark.parametrize("m", [1, 9, 80])
def test_qkv_of_rebuilt_8_bit_weights(m):
    """Bundles rebuilt into 8-bit blocks, projected, normed and rotated, against the same in float64 from the blocks."""
    I, D, R = 640, 64, 16
    x = randn((m, I), 1)
    ws = []
    for j, rows in enumerate((256, 128, 128)):
        ws.append(tb.reconstruct_weight_fp8((1 + 0.1 * randn((rows,), 2, 1.0, F32)).to(BF), randn((rows, I), 3 + j, 0.05),
                                            randn((rows, R), 6 + j, 0.05), randn((I, R), 9 + j, 0.05), tb.E8M0))
    wq, wk = randn((D,), 20), randn((D,), 21)
    pos, fr = torch.arange(5, 5 + m, device=DEV), frequencies(D)
    q, k, v = tb.qkv_forward(x, *ws, D, pos, fr, wq, wk)
    raw = [tb.dense_forward_fp8(x, *w) for w in ws]
    check(q, raw[0].view(m, -1, D), wq, pos, fr, 1e-6)
    check(k, raw[1].view(m, -1, D), wk, pos, fr, 1e-6)
    assert torch.equal(v, raw[2].view(m, -1, D))
    xq, xs = o.quantize_blocks(exact(x), 1, True)
    for got, w in zip((q, k), ws):
        y = o.block_product(xq, xs, w[0].cpu().double().numpy(), w[1].cpu().double().numpy())
        want = o.head_norm_rotate(y.reshape(m, -1, D), exact(wq if got is q else wk), pos.cpu().numpy(), fr.cpu().numpy(), 1e-6)
        # Two roundings to bf16 (2^-8 each), carried through a rotation of at most two terms.
        assert oracle.relative_frobenius_error(want.reshape(m, -1), exact(got.reshape(m, -1))) <= 2.0 ** -7
