"""Host-only refusals of the 8-bit integer calls, the residual norm and the rotation over several axes: the C ABI with
addresses that are never used, and the binding with CPU tensors."""

import ctypes

import pytest
import torch

tb = pytest.importorskip("rank_factored_linear_amd.binding")
lib = tb.lib
FAKE = 0x100000
INV, UNS = tb.TB_ERR_INVALID_ARGUMENT, tb.TB_ERR_UNSUPPORTED
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


def refused(fn, status, word):
    with pytest.raises(tb.TBError) as e:
        fn()
    assert e.value.status == status, str(e.value)
    assert word in str(e.value), str(e.value)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(q=None), INV), (dict(s=None), INV), (dict(m=-1), INV), (dict(i=0), INV), (dict(dt=2), INV),
    (dict(dt=3), INV), (dict(i=20), UNS), (dict(x=FAKE + 8), UNS), (dict(q=FAKE + 4), UNS), (dict(s=FAKE + 2), UNS),
    (dict(i=65544), UNS), (dict(m=1 << 31), UNS), (dict(m=0, x=None), 0),
])
def test_quantize_rows_int8_refuses(kw, status):
    a = dict(x=FAKE, q=FAKE, s=FAKE, m=4, i=256, dt=1)
    a.update(kw)
    assert lib.tb_quantize_rows_int8(a["x"], a["q"], a["s"], a["m"], a["i"], a["dt"], None) == status
    assert bool(lib.tb_last_error()) == (status != 0)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(ws=None), INV), (dict(y=None), INV), (dict(m=-1), INV),
    (dict(o=0), INV), (dict(i=0), INV), (dict(xd=2), INV), (dict(yd=3), INV), (dict(xs=FAKE), INV), (dict(xd=3), INV),
    (dict(i=8), UNS), (dict(i=24), UNS), (dict(x=FAKE + 8), UNS), (dict(w=FAKE + 8), UNS), (dict(y=FAKE + 1), UNS),
    (dict(ws=FAKE + 1), UNS), (dict(xd=3, xs=FAKE + 2), UNS), (dict(m=1 << 31), UNS), (dict(i=65552), UNS),
    (dict(o=1 << 31), UNS), (dict(m=1 << 24, o=1 << 20), UNS), (dict(m=0, x=None), 0),
])
def test_dense_forward_int8_refuses(kw, status):
    a = dict(x=FAKE, xs=None, w=FAKE, ws=FAKE, y=FAKE, m=4, o=64, i=64, xd=1, yd=1)
    a.update(kw)
    assert lib.tb_dense_forward_int8(a["x"], a["xs"], a["w"], a["ws"], a["y"], a["m"], a["o"], a["i"], a["xd"], a["yd"],
                                     None, 0, None) == status
    size = ctypes.c_size_t(77)
    if not {"x", "w", "ws", "y", "xs"} & set(kw) and status:
        if kw != dict(xd=3):
            assert lib.tb_dense_forward_int8_workspace_size(a["m"], a["o"], a["i"], a["xd"], a["yd"],
                                                            ctypes.byref(size)) == status
            assert size.value == 77


def test_binding_refuses_wrong_int8_operands():
    x, w, ws = torch.zeros(4, 384, dtype=BF), torch.zeros(256, 384, dtype=I8), torch.zeros(256)
    f = tb.dense_forward_int8
    refused(lambda: f(x, w, ws), INV, "GPU")                                  # well formed: only the device is wrong
    refused(lambda: f(x[:, :256], w, ws), INV, "Wq")
    refused(lambda: f(x, w.float(), ws), INV, "Wq")
    refused(lambda: f(x, w.to(torch.uint8), ws), INV, "Wq")
    refused(lambda: f(x, w, ws[:128]), INV, "w_scale")
    refused(lambda: f(x, w, ws.to(BF)), INV, "w_scale")
    refused(lambda: f(x.half(), w, ws), UNS, "float16")
    refused(lambda: f(x.to(I8), w, ws), INV, "x_scale")
    refused(lambda: f(x, w, ws, torch.zeros(4)), INV, "x_scale")
    refused(lambda: f(x.to(I8), w, ws, torch.zeros(5)), INV, "x_scale")
    refused(lambda: f(x, w, ws, out=torch.zeros(4, 255, dtype=BF)), INV, "out")
    refused(lambda: f(x, w, ws, out=torch.zeros(4, 256), out_dtype=BF), INV, "out")
    refused(lambda: f(x[0], w, ws), INV, "x must be")
    g = tb.quantize_rows_int8
    refused(lambda: g(x), INV, "GPU")
    refused(lambda: g(x[0]), INV, "x must be")
    refused(lambda: g(x.half()), UNS, "float16")
    refused(lambda: g(x, (torch.zeros(4, 384, dtype=torch.uint8), torch.zeros(4))), INV, "out")
    refused(lambda: g(x, (torch.zeros(4, 384, dtype=I8), torch.zeros(4, 1))), INV, "out")


# ---- residual norm ---------------------------------------------------------------------------------------------------

FAR = 1 << 24


def norm_call(m=4, n=64, scale=1.0, eps=1e-6, post=1, dt=1, hd=1, zd=1, st=0, tensors=True, **kw):
    a = dict(h=FAKE, y=FAKE + FAR, post_weight=FAKE + 2 * FAR, gate=FAKE + 3 * FAR, weight=FAKE + 4 * FAR,
             h_out=FAKE + 5 * FAR, z=FAKE + 6 * FAR, z_scale=None, h_stride=64, y_stride=64, h_out_stride=64, z_stride=64,
             gate_rows=4, gate_stride=0, gate_channels=1)
    a.update(kw)
    r = tb.Residual(**a)
    status = lib.tb_residual_norm(ctypes.byref(r) if tensors else None, m, n, scale, eps, 0.0, post, dt, hd, zd, st, None)
    return status, lib.tb_last_error().decode()


@pytest.mark.parametrize("kw,status,word", [
    (dict(tensors=False), INV, "tensors"), (dict(m=-1), INV, "m >= 0"), (dict(n=0), INV, "n >= 1"),
    (dict(m=1 << 25), UNS, "m exceeds"), (dict(n=32769), UNS, "n 32768"), (dict(eps=-1.0), INV, "eps"),
    (dict(eps=float("nan")), INV, "eps"), (dict(dt=2), INV, "dtype"), (dict(hd=3), INV, "dtype"),
    (dict(zd=0), INV, "z is in"), (dict(st=2), INV, "scale type"), (dict(h=None), INV, "h must"),
    (dict(y=None), INV, "go with a y"), (dict(y=None, gate=None, post=0, post_weight=None), INV, "together"),
    (dict(y=None, gate=None, post=0, post_weight=None, h_out=None, scale=0.5), INV, "go with a y"),
    (dict(h_out=None), INV, "together"), (dict(z=None), INV, "weight"), (dict(z=None, weight=None, zd=3), INV, "8 bits"),
    (dict(post=0), INV, "post_weight"), (dict(gate_rows=0), INV, "gate_rows"), (dict(gate_channels=2), INV, "gate_channels"),
    (dict(h_stride=-64), INV, "stride of h is"), (dict(h_out_stride=63), INV, "rows of h_out"),
    (dict(z_stride=32), INV, "rows of z"), (dict(y_stride=1 << 36), UNS, "stride of y"),
    (dict(gate_rows=1, gate_stride=-1), INV, "stride of gate"), (dict(h=FAKE + 1), UNS, "h must be aligned"),
    (dict(weight=FAKE + 1), UNS, "weight must"), (dict(z=FAKE + 1), UNS, "z must"),
    (dict(zd=3), INV, "z_scale"), (dict(z_scale=FAKE + 7 * FAR), INV, "z_scale"),
    (dict(zd=3, z_scale=FAKE + 7 * FAR, n=60), UNS, "n % 8"),
    (dict(zd=3, z_scale=FAKE + 7 * FAR + 2), UNS, "z_scale must"),
    (dict(zd=3, z_scale=FAKE + 7 * FAR, h=FAKE + 8), UNS, "16-byte"),
    (dict(zd=2, z_scale=FAKE + 7 * FAR, weight=FAKE + 2), UNS, "16-byte"),
    (dict(zd=2, z_scale=FAKE + 7 * FAR, y_stride=68), UNS, "16-byte"),
    (dict(zd=2, z_scale=FAKE + 7 * FAR, gate_rows=1, gate_stride=3), UNS, "16-byte"),
    (dict(h_out=FAKE + FAR), INV, "h_out overlaps y"), (dict(h_out=FAKE + 2), INV, "h_out overlaps h"),
    (dict(h_out=FAKE, h_out_stride=128), INV, "h_out overlaps h"), (dict(z=FAKE), INV, "z overlaps h"),
    (dict(z=FAKE + FAR, z_stride=66), INV, "z overlaps y"), (dict(z=FAKE + 5 * FAR), INV, "z overlaps h_out"),
    (dict(z=FAKE + FAR, zd=3, z_scale=FAKE + 7 * FAR), INV, "z overlaps y"),
    (dict(z=FAKE + 4 * FAR + 64), INV, "z overlaps weight"), (dict(h_out=FAKE + 3 * FAR), INV, "h_out overlaps gate"),
    (dict(zd=3, z_scale=FAKE + 6 * FAR + 16), INV, "z_scale overlaps z"),
    (dict(h_out=FAKE, hd=0, h_stride=32, h_out_stride=64), INV, "h_out overlaps h"),
    (dict(m=0, h=None), 0, ""),
])
def test_residual_norm_refuses(kw, status, word):
    got, message = norm_call(**kw)
    assert got == status, message
    assert word in message, message


def test_overlapping_rows_are_told_apart_at_one_stride():
    """Against sets of bytes: the last check passed is told by a refusal that comes behind it (a misplaced z_scale)."""
    n, m = 8, 3
    for stride in (8, 16, 20, 25):
        for shift in range(-60, 61):
            h = {1000 + t * stride + i for t in range(m) for i in range(n)}
            out = {1000 + shift + t * stride + i for t in range(m) for i in range(n)}
            status, message = norm_call(m=m, n=n, h=FAKE + 2000, h_out=FAKE + 2000 + 2 * shift, h_stride=stride,
                                        h_out_stride=stride, y_stride=n, z_stride=n, z=FAKE + 4 * FAR)
            assert status == INV
            if h.isdisjoint(out) and not -stride * m < shift < stride * m:
                assert "z overlaps weight" in message, (stride, shift)
            elif not h.isdisjoint(out) and shift:
                assert "h_out overlaps h" in message, (stride, shift)
            elif shift == 0:
                assert "z overlaps weight" in message
            else:   # between h's rows: apart, wherever each row is
                assert "z overlaps weight" in message or shift % stride and "h_out overlaps h" in message


def test_binding_refuses_wrong_norm_operands():
    h, y, w = torch.zeros(6, 64), torch.zeros(6, 64, dtype=BF), torch.zeros(64, dtype=BF)
    f = tb.residual_norm
    refused(lambda: f(h, y, w), INV, "GPU")
    refused(lambda: f(h[0], y, w), INV, "h must be")
    refused(lambda: f(h, y[:5], w), INV, "y must be")
    refused(lambda: f(h.half(), y, w), UNS, "float16")
    refused(lambda: f(h, y.half(), None), UNS, "float16")
    refused(lambda: f(h, y, w.float()), INV, "weight")
    refused(lambda: f(h, y, w[:32]), INV, "weight")
    refused(lambda: f(h, y, w, post_weight=w[:32], post_norm=True), INV, "post_weight")
    for g in ((5, 64), (4, 1), (6, 2), (64, 1), (6, 64, 1), (0, 64), (32,)):
        refused(lambda: f(h, y, w, gate=torch.zeros(g, dtype=BF)), INV, "gate")
    refused(lambda: f(h, y, w, gate=torch.zeros(64)), INV, "gate")
    refused(lambda: f(h, y, w, out_dtype=F32), UNS, "z is in")
    refused(lambda: f(h, y, w, out_dtype=tb.E4M3, scale_dtype=BF), UNS, "scales")
    refused(lambda: f(h, y, w, norm=False), INV, "go with the norm")
    refused(lambda: f(h, y, norm=False, out_dtype=I8), INV, "go with the norm")
    refused(lambda: f(h, y, w, outs=(h, y[:5])), INV, "out")
    refused(lambda: f(h, y, w, outs=(y, y)), INV, "out")
    refused(lambda: f(h, y, w, outs=(h, (y.to(I8), torch.zeros(5)))), INV, "out")
    refused(lambda: f(h, y, w, out_dtype=I8, outs=(h, y)), INV, "out")
    refused(lambda: f(h, None, w.float(), outs=(h, h)), INV, "without a y")
    refused(lambda: f(h, None, w.half()), UNS, "float16")


# ---- rotation over several axes --------------------------------------------------------------------------------------


def axes_call(pair_axis=(0,) * 8 + (1,) * 24, pairs=0, axes=2, norm=1, weight=FAKE, tokens=3, dim=64, rot=64, eps=1e-6,
              pos=FAKE, fr=FAKE, y=FAKE, n=1):
    arr = (tb.HeadPart * 1)(tb.HeadPart(FAKE, y, weight, 2, 128, 64, 128, 64))
    status = lib.tb_head_norm_rotate_axes(n, arr, tokens, dim, rot, pairs, axes, pos, None if pair_axis is None else
                                          bytes(pair_axis), fr, norm, eps, 0.0, 1, None)
    return status, lib.tb_last_error().decode()


@pytest.mark.parametrize("kw,status,word", [
    (dict(pairs=3), INV, "layout"), (dict(axes=0), INV, "axes"), (dict(axes=5), INV, "axes"), (dict(rot=0), INV, "rot_dim"),
    (dict(rot=3), INV, "rot_dim"), (dict(rot=66), INV, "rot_dim"), (dict(pair_axis=None), INV, "pair_axis"),
    (dict(pair_axis=(0,) * 31 + (2,)), INV, "pair 31"), (dict(pair_axis=(0, 1) * 16, pairs=2), INV, "consecutive"),
    (dict(norm=0), INV, "weight"), (dict(eps=-1.0), INV, "eps"), (dict(pos=None), INV, "positions"),
    (dict(fr=None), INV, "positions"), (dict(pos=FAKE + 4), UNS, "8-byte"), (dict(y=None), INV, "non-NULL"),
    (dict(n=0), INV, "n 0"), (dict(dim=1040), UNS, "head_dim"), (dict(tokens=0, weight=None, norm=0, eps=-1.0), 0, ""),
    (dict(tokens=0, pair_axis=(3,) * 32), INV, "pair 0"),
])
def test_rotation_over_axes_refuses(kw, status, word):
    got, message = axes_call(**kw)
    assert got == status, message
    assert word in message, message


def test_binding_refuses_wrong_axes():
    x, w = torch.zeros(5, 2, 64, dtype=BF), torch.zeros(64, dtype=BF)
    pos, fr = torch.zeros(3, 5, dtype=torch.int64), torch.zeros(32, dtype=torch.float64)
    f = lambda pos=pos, fr=fr, axes=(0, 1, 2, 2) * 8, w=w, **kw: tb.head_norm_rotate([(x, w)], pos, fr, axes=axes, **kw)   # noqa: E731
    refused(lambda: f(), INV, "GPU")
    refused(lambda: f(axes=[0, 1, 2, 2] * 8), INV, "GPU")
    refused(lambda: f(axes=(0,) * 31), INV, "31")
    refused(lambda: f(axes=(0,) * 31 + (3,)), INV, "outside")
    refused(lambda: f(axes=(0,) * 31 + (-1,)), INV, "outside")
    refused(lambda: f(pos=pos[0]), INV, "positions")
    refused(lambda: f(pos=torch.zeros(5, 5, dtype=torch.int64)), INV, "positions")
    refused(lambda: f(pos=pos[:, :4]), INV, "positions")
    refused(lambda: f(pos=pos.int()), INV, "positions")
    refused(lambda: f(pos=None, fr=None), INV, "axes go with")
    refused(lambda: f(axes=None, pos=pos[0], norm=False), INV, "go with axes")
    refused(lambda: f(axes=None, pos=pos[0], axis_halves=True), INV, "go with axes")
    refused(lambda: f(axis_halves=True), INV, "consecutive")
    refused(lambda: f(axes=(0,) * 32, axis_halves=True, interleaved=True), INV, "not both")


# ---- the path that ends in them --------------------------------------------------------------------------------------


def channels(out, n=64):
    return torch.zeros(out, n, dtype=I8), torch.zeros(out)


def test_qkv_checks_int8_before_the_first_launch():
    x = torch.zeros(3, 64, dtype=BF)
    x8 = torch.zeros(3, 64, dtype=I8), torch.zeros(3)

    def call(q=channels(256), k=channels(64), v=channels(64), x=x, dim=64, pos=None, fr=None, **more):
        return lambda: tb.qkv_forward(x, q, k, v, dim, pos, fr, **more)

    refused(call(), INV, "GPU")
    refused(call(x=x8), INV, "GPU")
    refused(call(x=x8, out_dtype=F32), INV, "GPU")
    refused(call(k=(torch.zeros(64, 64, dtype=tb.E4M3), torch.zeros(1, 1))), INV, "Wq")
    refused(call(v=(channels(64)[0], torch.zeros(64, 1))), INV, "w_scale")
    refused(call(x=(x8[0], torch.zeros(4))), INV, "x_scale")
    refused(call(x=(x8[0].to(tb.E4M3), x8[1])), UNS, "float8")
    refused(call(x=(x, x8[1])), INV, "x_scale")
    refused(call(x=x, out_dtype=F32), INV, "heads of an x")
    refused(call(x=x8, out_dtype=torch.float16), UNS, "float16")
    refused(call(x=x8 + x8), INV, "numbers, scales")
    refused(call(x=x8, q_weight=torch.zeros(64)), INV, "head weight")
    n8 = torch.zeros(3, 72, dtype=BF)
    refused(call(channels(256, 72), channels(64, 72), channels(64, 72), n8), UNS, "multiple of 16")
    pos, fr = torch.zeros(2, 3, dtype=torch.int64), torch.zeros(32, dtype=torch.float64)
    refused(call(pos=pos, fr=fr, axes=(0, 1) * 16), INV, "GPU")
    refused(call(pos=pos, fr=fr, axes=(0, 1) * 16, axis_halves=True), INV, "consecutive")
    refused(call(pos=pos, fr=fr, axes=(0, 2) * 16), INV, "outside")
    refused(call(pos=pos, fr=fr), INV, "positions")
    bundle = torch.zeros(64, dtype=BF), torch.zeros(64, 64, dtype=BF), None, None
    refused(call(bundle, bundle, bundle, x=x8), INV, "8 bits")
