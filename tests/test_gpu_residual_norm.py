"""The norms before and after a block on the GPU against the float64 oracle, and the run of calls that they stand in.

Tolerance, with u = 2^-23 for each fp32 operation.  A norm's factor r comes from a sum of n squares (gamma(n), halved by
the root) and four operations.  a = y r (w + offset) gate: r and four more.  h' = scale h + a: two on |scale h| + |a|; it
is rounded once to be stored.  z = h' r' (w + offset) inherits h's error dh (times |w + offset| / rms, and through the rms
at most its norm over h's) and adds r' and three operations; it is rounded once, by half a step of its type:
  bf16 2^-8 of the value, fp32 2^-24;
  int8 half of its row's scale, which is off by what the largest z is, over 127, and two operations;
  e4m3 2^-4 of the value or 2^-10 of the scale; the scale is off by what the block's largest z is, over 448, or is the
  power of two on either side of it.
"""

import numpy as np
import pytest
import torch

from oracle import serving as o
from parity_util import exact, gamma

pytestmark = pytest.mark.gpu

tb = pytest.importorskip("rank_factored_linear_amd.binding")
DEV = "cuda"
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8
U = 2.0 ** -23


def randn(shape, seed, sd=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * sd).to(dtype).to(DEV)


def half_step(dtype):
    return 2.0 ** -8 if dtype == BF else 2.0 ** -24


def spread_gate(gate, m, n):
    if gate is None:
        return None
    g = exact(gate)
    g = g[None] if g.ndim == 1 else g
    return np.broadcast_to(np.repeat(g, m // g.shape[0], 0), (m, n))


def check(got, h, y=None, weight=None, post_norm=False, post_weight=None, gate=None, residual_scale=1.0, eps=1e-6,
          weight_offset=0.0):
    ho, z = got
    e = lambda t: None if t is None else exact(t)   # noqa: E731
    H, Y, W, P = e(h), e(y), e(weight), e(post_weight)
    m, n = H.shape
    G = spread_gate(gate, m, n)
    want_h, want_z, a = o.residual_norm(H, Y, W, post_norm, P, G, residual_scale, eps, weight_offset)
    # gate and weight may cancel (w + offset near zero): their sum is off by u of its terms.
    fuzz = np.zeros_like(H)
    if post_norm and P is not None:
        base = Y / np.sqrt(np.mean(Y ** 2, axis=1, keepdims=True) + eps)
        fuzz = U * np.abs(base * (1 if G is None else G)) * (np.abs(P) + abs(weight_offset))
    dh = np.abs(a) * (gamma(n) / 2 + 8 * U) + fuzz + 2 * U * (np.abs(residual_scale * H) + np.abs(a)) if y is not None \
        else np.zeros_like(H)
    if y is None:
        assert ho is h
    else:
        room = dh + half_step(ho.dtype) * (np.abs(want_h) + dh)
        err = np.abs(exact(ho) - want_h) - room
        assert (err <= 0).all(), ("h", float(err.max()))
    if z is None:
        return
    rms = np.sqrt(np.mean(want_h ** 2, axis=1, keepdims=True) + eps)
    w = np.ones(n) if W is None else np.abs(W + weight_offset)
    wsize = np.ones(n) if W is None else np.abs(W) + abs(weight_offset)
    norm = np.sqrt((want_h ** 2).sum(1, keepdims=True))
    through = np.divide(np.sqrt((dh ** 2).sum(1, keepdims=True)), norm, out=np.zeros_like(norm), where=norm > 0)
    dz = w / rms * dh + np.abs(want_z) * (through + gamma(n) / 2 + 8 * U) + U * np.abs(want_h) / rms * wsize
    if isinstance(z, tuple):
        q, s = z[0].cpu().double().numpy(), z[1].cpu().double().numpy()
        top_off = dz.max(1)
        if z[0].dtype == I8:
            assert np.isfinite(s).all()
            top = np.maximum(np.abs(want_z).max(1), 2.0 ** -100)
            assert (np.abs(s - top / 127) <= top_off / 127 + 2 * U * s).all()
            assert np.abs(q).max() <= 127 and (q == np.rint(q)).all()
            err = np.abs(q * s[:, None] - want_z) - (s[:, None] / 2 + dz + 4 * U * np.abs(want_z))
        else:
            blocks = s.shape[1]
            big, off = np.zeros((m, blocks * 128)), np.zeros((m, blocks * 128))
            big[:, :n], off[:, :n] = np.abs(want_z), dz
            top, off = big.reshape(m, blocks, 128).max(2), off.reshape(m, blocks, 128).max(2)
            if z[1].dtype == tb.E8M0:
                assert np.array_equal(np.log2(s), np.round(np.log2(s)))
                assert (448 * s >= top - off).all() and ((448 * s / 2 < top + off) | (s == 2.0 ** -127)).all()
            else:
                top = np.maximum(top, 2.0 ** -100)
                assert (np.abs(s - top / 448) <= off / 448 + 2 * U * s).all()
            sp = np.repeat(s, 128, 1)[:, :n]
            half = np.maximum(2.0 ** -4 * (np.abs(want_z) + dz), 2.0 ** -10 * sp)
            err = np.abs(q * sp - want_z) - (half + dz + 5 * U * np.abs(want_z))
        assert (err <= 0).all(), ("z", float(err.max()))
        return
    err = np.abs(exact(z) - want_z) - (dz + half_step(z.dtype) * (np.abs(want_z) + dz))
    assert (err <= 0).all(), ("z", float(err.max()))


SIZES = [(1, 1), (1, 8), (3, 2), (2, 7), (5, 64), (4, 65), (3, 130), (7, 264), (2, 1152), (3, 1155), (5, 2048), (2, 2056),
         (2, 4099), (3, 5376), (2, 8192), (2, 8200), (1, 9001), (2, 16384), (1, 16400), (1, 32768), (1, 32767)]


def inputs(m, n, dtype, stream):
    return dict(h=randn((m, n), 1, 3.0, stream), y=randn((m, n), 2, 0.5, dtype), weight=randn((n,), 3, 0.2, dtype),
                post_weight=randn((n,), 4, 0.2, dtype))


@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n", SIZES)
def test_parity(m, n, dtype, stream):
    print(m, n, dtype, stream, flush=True)
    a = inputs(m, n, dtype, stream)
    for kw in (dict(a, post_norm=True, gate=randn((n,), 5, 1.0, dtype), weight_offset=1.0, residual_scale=0.7),
               dict(h=a["h"], y=a["y"], weight=a["weight"], gate=randn((m, 1), 6, 1.0, dtype)),
               dict(h=a["h"], y=a["y"], post_norm=True, eps=1e-3),
               dict(h=a["h"], y=a["y"], weight=a["weight"], gate=randn((m, n), 7, 1.0, dtype), residual_scale=-1.5)):
        check(tb.residual_norm(**kw), **kw)
    if stream == dtype:
        kw = dict(h=a["h"], weight=a["weight"], weight_offset=1.0)
        check(tb.residual_norm(**kw), **kw)


@pytest.mark.parametrize("held", ["int8", "f32", "e8m0"])
@pytest.mark.parametrize("dtype,stream", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("m,n", [(m, n) for m, n in SIZES if n % 8 == 0])
def test_8_bit_results(m, n, dtype, stream, held):
    print(m, n, dtype, stream, held, flush=True)
    a = inputs(m, n, dtype, stream)
    kind = dict(out_dtype=I8 if held == "int8" else tb.E4M3, scale_dtype=tb.E8M0 if held == "e8m0" else F32)
    for kw in (dict(a, post_norm=True, gate=randn((n,), 5, 1.0, dtype), weight_offset=1.0),
               dict(h=a["h"], y=a["y"], weight=a["weight"])):
        got = tb.residual_norm(**kw, **kind)
        check(got, **kw)
        h_alone, none = tb.residual_norm(**{k: v for k, v in kw.items() if k != "weight"}, norm=False)
        assert none is None and torch.equal(got[0], h_alone)


@pytest.mark.parametrize("groups", [1, 2, 3, 6])
@pytest.mark.parametrize("n", [264, 77])
def test_gates_of_groups(n, groups):
    a = inputs(6, n, BF, BF)
    for width in (n, 1):
        kw = dict(h=a["h"], y=a["y"], weight=a["weight"], gate=randn((groups, width), 5))
        check(tb.residual_norm(**kw), **kw)
        wide = torch.zeros(groups, 2 * n, dtype=BF, device=DEV)   # a strided gate
        wide[:, n:n + width] = kw["gate"]
        got = tb.residual_norm(**{**kw, "gate": wide[:, n:n + width]})
        want = tb.residual_norm(**kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("n,pad", [(264, 8), (264, 3), (77, 1)])
def test_strides_and_in_place(n, pad):
    """Views of wider rows in and out, h' over h and z over y; what lies beside them stays."""
    m = 5
    wide = lambda seed: randn((m, 2 * n + pad), seed)   # noqa: E731
    H, Y = wide(1), wide(2)
    w, g = randn((n,), 3), randn((n,), 4)
    kw = dict(weight=w, gate=g, post_norm=True)
    want = tb.residual_norm(H[:, :n].contiguous(), Y[:, n:2 * n].contiguous(), **kw)
    got = tb.residual_norm(H[:, :n], Y[:, n:2 * n], **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # Both outputs as two halves of one buffer: their rows interleave.
    O = torch.full((m, 2 * n + pad), 9.0, dtype=BF, device=DEV)
    tb.residual_norm(H[:, :n], Y[:, n:2 * n], **kw, outs=(O[:, :n], O[:, n:2 * n]))
    assert torch.equal(O[:, :n], want[0]) and torch.equal(O[:, n:2 * n], want[1]) and (O[:, 2 * n:] == 9).all()
    keep_h, keep_y = H.clone(), Y.clone()
    tb.residual_norm(H[:, :n], Y[:, n:2 * n], **kw, outs=(H[:, :n], Y[:, n:2 * n]))
    assert torch.equal(H[:, :n], want[0]) and torch.equal(Y[:, n:2 * n], want[1])
    assert torch.equal(H[:, n:], keep_h[:, n:]) and torch.equal(Y[:, :n], keep_y[:, :n])
    assert torch.equal(Y[:, 2 * n:], keep_y[:, 2 * n:])


def test_many_rows_and_determinism():
    for n in (72, 1152):
        m = 5003
        a = inputs(m, n, BF, F32)
        kw = dict(a, post_norm=True, gate=randn((n,), 5), weight_offset=1.0)
        got = tb.residual_norm(**kw)
        check(got, **kw)
        again = tb.residual_norm(**kw)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
        one = tb.residual_norm(**{**kw, "h": a["h"][77:78], "y": a["y"][77:78]})
        assert torch.equal(one[0][0], got[0][77]) and torch.equal(one[1][0], got[1][77])


@pytest.mark.parametrize("held", [None, I8, "e4m3"])
def test_rows_that_are_not_finite_stay_alone(held):
    n = 264
    a = inputs(4, n, BF, BF)
    a["y"][1, 5] = float("nan")
    a["h"][2, 7] = float("inf")
    clean = inputs(4, n, BF, BF)
    kw = dict(post_norm=True, out_dtype=tb.E4M3 if held == "e4m3" else held)
    ho, z = tb.residual_norm(**a, **kw)
    hc, zc = tb.residual_norm(**clean, **kw)
    flat = lambda v: v[0].float() * (v[1][:, None] if held == I8 else v[1].repeat_interleave(128, 1)[:, :n]) \
        if isinstance(v, tuple) else v.float()   # noqa: E731
    assert torch.equal(ho[[0, 3]], hc[[0, 3]]) and torch.equal(flat(z)[[0, 3]], flat(zc)[[0, 3]])
    assert ho[1].isnan().all() and flat(z)[1].isnan().all()
    assert ho[2, 7].isinf() and ho[2, :7].isfinite().all()
    # inf / inf at the one place (and the whole scale behind it), finite / inf elsewhere
    assert flat(z)[2, 7].isnan()
    if held is None:
        assert (z[2, :7] == 0).all() and (z[2, 8:] == 0).all()
    elif held == I8:
        assert z[1][2].isnan() and (z[0][2] == 0).all()
    else:
        assert z[1][2, 0].isnan() and (flat(z)[2, 128:] == 0).all()


def test_zero_rows_and_no_rows():
    n = 264
    h, y = torch.zeros(3, n, dtype=BF, device=DEV), torch.zeros(3, n, dtype=BF, device=DEV)
    for out in (None, I8, tb.E4M3):
        ho, z = tb.residual_norm(h, y, post_norm=True, out_dtype=out)
        assert (ho == 0).all() and ((z if out is None else z[0].float()) == 0).all()
        ho, z = tb.residual_norm(h[:0], y[:0], post_norm=True, out_dtype=out, gate=torch.ones(0, 1, dtype=BF, device=DEV))
        assert ho.shape == (0, n) and (z if out is None else z[0]).shape == (0, n)


def test_another_stream_and_a_graph():
    a, b = inputs(9, 1152, BF, BF), inputs(9, 1152, BF, BF)
    b["h"] = b["h"] * 2 + 1
    kw = dict(post_norm=True, out_dtype=I8)
    want = [tb.residual_norm(**x, **kw) for x in (a, b)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = tb.residual_norm(**b, **kw)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[1][0]) and torch.equal(got[1][0], want[1][1][0])
    h = a["h"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tb.residual_norm(**{**a, "h": h}, **kw)
    for k in range(4):
        h.copy_((a, b)[k % 2]["h"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[k % 2][0]) and torch.equal(out[1][0], want[k % 2][1][0])
        assert torch.equal(tb.residual_norm(**a, **kw)[0], want[0][0])


# --------------------------------------------------------------------------------------------------------------------
# The run of calls: residual norm into 8 bits, projections, head norms and rotation, the block's projection, the next norm
# --------------------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("m", [1, 9, 70])
def test_a_layer_in_8_bits(m, kind):
    n, D, hq, hk = 256, 64, 4, 2
    make = tb.quantize_weight_int8 if kind == "int8" else tb.quantize_weight
    q, k, v = (make(randn((r * D, n), r, 0.06)) for r in (hq, hk, 3))
    proj = make(randn((n, hq * D), 9, 0.06))
    h, y, w = randn((m, n), 1, 2.0, F32), randn((m, n), 2), randn((n,), 3, 0.1)
    pos = torch.stack([torch.arange(m, device=DEV) + 3 * a for a in range(3)])
    axes = (0,) * 8 + (1,) * 12 + (2,) * 12
    fr = 1e4 ** (-torch.arange(32, dtype=torch.float64) / 32).to(DEV)
    wq, wk = randn((D,), 4, 0.1), randn((D,), 5, 0.1)
    out = I8 if kind == "int8" else tb.E4M3
    h1, x8 = tb.residual_norm(h, y, w, post_norm=True, weight_offset=1.0, out_dtype=out)
    Q, K, V = tb.qkv_forward(x8, q, k, v, D, pos, fr, wq, wk, weight_offset=1.0, axes=axes)
    # Each call by itself, the same bits.
    dense = tb.dense_forward_int8 if kind == "int8" else tb.dense_forward_fp8
    parts = [dense(x8[0], *p, x_scale=x8[1]).view(m, -1, D) for p in (q, k, v)]
    Q2, K2 = tb.head_norm_rotate([(parts[0], wq), (parts[1], wk)], pos, fr, weight_offset=1.0, axes=axes)
    assert torch.equal(Q, Q2) and torch.equal(K, K2) and torch.equal(V, parts[2]) and Q.dtype == BF
    # The wide x gives the same where it is quantised in the call from the same values.
    wide = (x8[0].float() * x8[1][:, None]).to(BF) if kind == "int8" else None
    if wide is not None:
        again = tb.qkv_forward(wide, q, k, v, D, pos, fr, wq, wk, weight_offset=1.0, axes=axes)
        x8w = tb.quantize_rows_int8(wide)
        assert torch.equal(again[2], dense(x8w[0], *v, x_scale=x8w[1]).view(m, -1, D))
    block = dense(Q.reshape(m, -1), *proj)
    h2, z = tb.residual_norm(h1, block, w, post_norm=True, gate=randn((n,), 6, 1.0), weight_offset=1.0, outs=(h1, block))
    assert h2 is h1 and z is block and h2.isfinite().all() and z.isfinite().all()
    assert abs(float(z.float().pow(2).mean()) - 1) < 0.5   # normed rows, weights near one


@pytest.mark.parametrize("held", [None, I8, "e4m3"])
@pytest.mark.parametrize("dtype,stream", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("n", [72, 77, 1152, 1155, 2056, 5376, 8192])
def test_a_row_is_the_same_in_any_batch(n, dtype, stream, held):
    """However many rows there are, which decides how many threads hold one."""
    if held is not None and n % 8:
        pytest.skip("8-bit results need rows of eights")
    m = 2100
    a = inputs(m, n, dtype, stream)
    kw = dict(weight=a["weight"], post_weight=a["post_weight"], post_norm=True, gate=randn((n,), 5, 1.0, dtype),
              weight_offset=1.0, residual_scale=0.7, out_dtype=tb.E4M3 if held == "e4m3" else held)
    flat = lambda z: [z] if held is None else [t.float() for t in z]   # noqa: E731
    ho, z = tb.residual_norm(a["h"], a["y"], **kw)
    for first, k in ((0, 1), (7, 3), (2, 300), (1000, 600), (11, 1100)):
        h1, z1 = tb.residual_norm(a["h"][first:first + k], a["y"][first:first + k], **kw)
        assert torch.equal(h1, ho[first:first + k]), k
        assert all(torch.equal(p, q[first:first + k]) for p, q in zip(flat(z1), flat(z))), k


@pytest.mark.parametrize("n", [264, 1155, 5376])
def test_the_first_norm_of_a_residual_in_fp32(n):
    """No block before it: z in the type of the weight, of out_dtype, or of the residual; 8 bits from either."""
    h, w = randn((5, n), 1, 3.0, F32), randn((n,), 2, 0.2)
    for kw, dtype in ((dict(weight=w, weight_offset=1.0), BF), (dict(weight=w.float()), F32), (dict(), F32)):
        got = tb.residual_norm(h, **kw)
        assert got[1].dtype == dtype
        check(got, h, **kw)
    got = tb.residual_norm(h, out_dtype=BF)
    assert got[1].dtype == BF
    check(got, h)
    if n % 8 == 0:
        for weight in (w, None):
            for kind in (I8, tb.E4M3):
                check(tb.residual_norm(h, None, weight, out_dtype=kind), h, None, weight)


def test_a_single_row_takes_any_stride():
    """The stride between rows that a tensor of one row reports is not looked at."""
    w, big = randn((264,), 3), randn((40, 264), 1)
    h = big.as_strided((1, 264), (7, 1))
    want = tb.residual_norm(h.contiguous(), big[3:4], w)
    got = tb.residual_norm(h, big.as_strided((1, 264), (1 << 40, 1), 3 * 264), w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def off_by(t, offset, pad):
    """(t's values `offset` elements into a buffer of NaN, rows `pad` apart beyond their length; the buffer)"""
    m, n = (1, len(t)) if t.dim() == 1 else t.shape
    big = torch.full((offset + m * (n + pad) + 8,), float("nan"), dtype=t.dtype, device=DEV)
    view = big.as_strided((m, n), (n + pad, 1), offset)
    view.copy_(t.view(m, n))
    return (view[0] if t.dim() == 1 else view), big


def untouched(big, offset, m, n, pad):
    inside = torch.zeros(len(big), dtype=torch.bool, device=DEV)
    inside.as_strided((m, n), (n + pad, 1), offset).fill_(True)
    return bool(big[~inside].isnan().all()) and not bool(big[inside].isnan().any())


@pytest.mark.parametrize("dtype,stream", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("n", [1, 5, 7, 8, 9, 10, 11, 12, 13, 14, 15, 264, 519, 1157, 5376, 5377, 8199, 16391, 24579, 32766])
def test_rows_at_any_address(n, dtype, stream):
    """Rows whose length, stride and address fit no 16 bytes, NaN around them: nothing of the neighbours' comes in or is
    written, also in place, and a row has the bits that it has elsewhere."""
    m, pad = 5, 3
    at = dict(h=1, y=2, weight=3, post_weight=5, gate=7)
    given = dict(inputs(m, n, dtype, stream), gate=randn((m, n), 9, 0.5, dtype))
    kw = dict(post_norm=True, residual_scale=0.7, weight_offset=1.0)
    v = {k: off_by(t, at[k], 0 if t.dim() == 1 else pad) for k, t in given.items()}
    views = {k: t[0] for k, t in v.items()}
    out_h, big_h = off_by(torch.zeros(m, n, dtype=stream), 3, pad)
    out_z, big_z = off_by(torch.zeros(m, n, dtype=dtype), 1, pad)
    got = tb.residual_norm(**views, **kw, outs=(out_h, out_z))
    assert got[0] is out_h and got[1] is out_z
    check(got, **given, **kw)
    assert untouched(big_h, 3, m, n, pad) and untouched(big_z, 1, m, n, pad)
    want = tb.residual_norm(**given, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    tb.residual_norm(**views, **kw, outs=(views["h"], views["y"]))
    assert torch.equal(views["h"], want[0]) and torch.equal(views["y"], want[1])
    assert untouched(v["h"][1], 1, m, n, pad) and untouched(v["y"][1], 2, m, n, pad)
