"""Host-only refusals of the 8-bit and head-norm entry points: the C ABI with addresses that are never used, and the
binding with CPU tensors (shape and dtype checks come before the device checks)."""

import ctypes

import pytest
import torch

tb = pytest.importorskip("rank_factored_linear_amd.binding")
lib = tb.lib
FAKE = 0x100000
INV, UNS = tb.TB_ERR_INVALID_ARGUMENT, tb.TB_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(q=None), INV), (dict(s=None), INV), (dict(m=-1), INV), (dict(i=0), INV),
    (dict(dt=2), INV), (dict(st=2), INV), (dict(i=20), UNS), (dict(x=FAKE + 8), UNS), (dict(q=FAKE + 4), UNS),
    (dict(s=FAKE + 2), UNS), (dict(i=(1 << 25) + 8), UNS), (dict(m=1 << 31), UNS), (dict(m=0, x=None), 0),
])
def test_quantize_activations_refuses(kw, status):
    a = dict(x=FAKE, q=FAKE, s=FAKE, m=4, i=256, dt=1, st=0)
    a.update(kw)
    assert lib.tb_quantize_activations(a["x"], a["q"], a["s"], a["m"], a["i"], a["dt"], a["st"], None) == status
    assert bool(lib.tb_last_error()) == (status != 0)


@pytest.mark.parametrize("kw,status", [
    (dict(w0=None), INV), (dict(q=None), INV), (dict(sc=None), INV), (dict(u=None), INV), (dict(v=None), INV),
    (dict(o=0), INV), (dict(i=0), INV), (dict(r=-1), INV), (dict(dt=5), INV), (dict(st=-1), INV), (dict(i=12), UNS),
    (dict(w0=FAKE + 8), UNS), (dict(u=FAKE + 8), UNS), (dict(q=FAKE + 8), UNS), (dict(s=FAKE + 1), UNS),
    (dict(o=1 << 31), UNS), (dict(o=1 << 30, i=1 << 25), UNS),
])
def test_reconstruct_weight_fp8_refuses(kw, status):
    a = dict(s=FAKE, w0=FAKE, u=FAKE, v=FAKE, q=FAKE, sc=FAKE, o=64, i=64, r=8, dt=1, st=1)
    a.update(kw)
    assert lib.tb_reconstruct_weight_fp8(a["s"], a["w0"], a["u"], a["v"], a["q"], a["sc"], a["o"], a["i"], a["r"],
                                         a["dt"], a["st"], None) == status
    assert lib.tb_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(ws=None), INV), (dict(y=None), INV), (dict(m=-1), INV),
    (dict(o=0), INV), (dict(i=0), INV), (dict(xd=3), INV), (dict(yd=2), INV), (dict(st=2), INV),
    (dict(xs=FAKE), INV),                 # scales with an x that is not in e4m3
    (dict(xd=2), INV),                    # an e4m3 x without scales
    (dict(i=8), UNS), (dict(i=24), UNS), (dict(x=FAKE + 8), UNS), (dict(w=FAKE + 8), UNS), (dict(y=FAKE + 1), UNS),
    (dict(ws=FAKE + 1), UNS), (dict(xd=2, xs=FAKE + 2), UNS), (dict(m=1 << 31), UNS), (dict(i=1 << 26), UNS),
    (dict(m=0, x=None), 0),
])
def test_dense_forward_fp8_refuses(kw, status):
    a = dict(x=FAKE, xs=None, w=FAKE, ws=FAKE, y=FAKE, m=4, o=64, i=64, xd=1, yd=1, st=0)
    a.update(kw)
    assert lib.tb_dense_forward_fp8(a["x"], a["xs"], a["w"], a["ws"], a["y"], a["m"], a["o"], a["i"], a["xd"], a["yd"],
                                    a["st"], None, 0, None) == status


def _parts(*parts):
    arr = (tb.HeadPart * len(parts))()
    for j, p in enumerate(parts):
        a = dict(x=FAKE, y=FAKE, w=FAKE, h=2, xt=128, xh=64, yt=128, yh=64)
        a.update(p)
        arr[j] = tb.HeadPart(a["x"], a["y"], a["w"], a["h"], a["xt"], a["xh"], a["yt"], a["yh"])
    return arr


@pytest.mark.parametrize("part,kw,status", [
    (dict(x=None), {}, INV), (dict(y=None), {}, INV), (dict(h=-1), {}, INV), (dict(xt=-128), {}, INV),
    (dict(yt=64), {}, INV),               # tokens overlap
    (dict(yh=32), {}, INV),               # heads overlap
    (dict(yt=0, yh=0), {}, INV), (dict(yt=96, yh=64), {}, INV),
    ({}, dict(n=0), INV), ({}, dict(n=9), INV), ({}, dict(t=-1), INV), ({}, dict(d=0), INV), ({}, dict(r=3), INV),
    ({}, dict(r=66), INV), ({}, dict(r=-2), INV), ({}, dict(eps=-1.0), INV), ({}, dict(eps=float("nan")), INV),
    ({}, dict(dt=2), INV), ({}, dict(pos=None), INV), ({}, dict(fr=None), INV), ({}, dict(parts=None), INV),
    ({}, dict(d=1032), UNS), (dict(h=1 << 16), {}, UNS), (dict(x=FAKE + 1), {}, UNS), (dict(w=FAKE + 1), {}, UNS),
    ({}, dict(pos=FAKE + 4), UNS), ({}, dict(t=1 << 31), UNS), (dict(xt=1 << 41), {}, UNS),
    ({}, dict(t=0, pos=None), 0), (dict(h=0, x=None), {}, 0),
])
def test_head_norm_rotate_refuses(part, kw, status):
    a = dict(n=1, t=3, d=64, r=64, inter=0, pos=FAKE, fr=FAKE, eps=1e-6, dt=1, parts=_parts(part))
    a.update(kw)
    assert lib.tb_head_norm_rotate(a["n"], a["parts"], a["t"], a["d"], a["r"], a["inter"], a["pos"], a["fr"], a["eps"],
                                   0.0, a["dt"], None) == status


def test_parts_that_write_into_each_other_are_refused():
    call = lambda *parts: lib.tb_head_norm_rotate(len(parts), _parts(*parts), 3, 64, 64, 0, FAKE, FAKE, 1e-6,   # noqa: E731
                                                  0.0, 1, None)
    far = dict(x=FAKE << 1, y=FAKE << 2)
    assert call(far, dict(x=FAKE << 3, y=FAKE << 2)) == INV      # one output for both
    assert call(far, dict(x=FAKE << 2, y=FAKE << 3)) == INV      # the first writes what the second reads
    assert call(far, dict(x=FAKE << 3, y=FAKE << 1)) == INV
    assert call(dict(xt=256)) == INV                             # in place, but rows elsewhere
    assert call(dict(xh=128, xt=256)) == INV


def test_a_bad_second_part_is_refused():
    arr = _parts({}, dict(y=None))
    assert lib.tb_head_norm_rotate(2, arr, 3, 64, 64, 0, FAKE, FAKE, 1e-6, 0.0, 1, None) == INV


def _raises(fn, status, word):
    with pytest.raises(tb.TBError) as e:
        fn()
    assert e.value.status == status, str(e.value)
    assert word in str(e.value), str(e.value)


BF = torch.bfloat16


def _dense(m=4, o=256, i=384, scale=torch.float32, dtype=BF):
    return (torch.zeros(m, i, dtype=dtype), torch.zeros(o, i, dtype=tb.E4M3),
            torch.zeros(-(-o // 128), -(-i // 128), dtype=scale))


def test_binding_refuses_wrong_dense_operands():
    x, w, ws = _dense()
    f = tb.dense_forward_fp8
    _raises(lambda: f(x, w, ws), INV, "GPU")                                  # well formed: only the device is wrong
    _raises(lambda: f(x[:, :256], w, ws), INV, "Wq")
    _raises(lambda: f(x, w.view(torch.uint8), ws), INV, "Wq")
    _raises(lambda: f(x, w, ws[:1]), INV, "w_scale")
    _raises(lambda: f(x, w, ws.to(BF)), UNS, "scales")
    _raises(lambda: f(x, w, ws, x_scale=torch.zeros(4, 3)), INV, "x_scale")
    xq = torch.zeros(4, 384, dtype=tb.E4M3)
    _raises(lambda: f(xq, w, ws), INV, "x_scale")
    _raises(lambda: f(xq, w, ws, x_scale=torch.zeros(4, 2)), INV, "x_scale")
    _raises(lambda: f(xq, w, ws, x_scale=torch.zeros(4, 3, dtype=tb.E8M0)), INV, "x_scale")
    _raises(lambda: f(x, w, ws, out=torch.zeros(4, 255, dtype=BF)), INV, "out")
    _raises(lambda: f(x, w, ws, out=torch.zeros(4, 256, dtype=BF), out_dtype=torch.float32), INV, "out")
    _raises(lambda: f(x.half(), w, ws), UNS, "float16")
    _raises(lambda: f(x, w, ws, out_dtype=torch.float16), UNS, "float16")
    _raises(lambda: f(x[0], w, ws), INV, "x must be")


def test_binding_refuses_wrong_rebuild_operands():
    s, W0, U, V = (torch.zeros(*n, dtype=BF) for n in ((256,), (256, 64), (256, 8), (64, 8)))
    f = tb.reconstruct_weight_fp8
    _raises(lambda: f(s, W0, U, V), INV, "GPU")
    _raises(lambda: f(s[:8], W0, U, V), INV, "s")
    _raises(lambda: f(s, W0, U[:8], V), INV, "U")
    _raises(lambda: f(s, W0, U, None), INV, "together")
    _raises(lambda: f(None, W0[0], None, None), INV, "W0")
    _raises(lambda: f(s, W0, U, V, scale_dtype=BF), UNS, "scales")
    q, sc = torch.zeros(256, 64, dtype=tb.E4M3), torch.zeros(2, 1)
    _raises(lambda: f(s, W0, U, V, out=(q, sc[:1])), INV, "out")
    _raises(lambda: f(s, W0, U, V, out=(q[:, :8], sc)), INV, "out")
    _raises(lambda: tb.quantize_weight(W0), INV, "GPU")
    _raises(lambda: tb.quantize_activations(W0), INV, "GPU")
    _raises(lambda: tb.quantize_activations(W0, torch.float16), UNS, "scales")
    _raises(lambda: tb.quantize_activations(W0[0]), INV, "x must be")


def test_binding_refuses_wrong_heads():
    q, k, w = torch.zeros(3, 4, 64, dtype=BF), torch.zeros(3, 1, 64, dtype=BF), torch.zeros(64, dtype=BF)
    pos, fr = torch.arange(3), torch.zeros(32, dtype=torch.float64)
    f = tb.head_norm_rotate
    _raises(lambda: f([(q, w), (k, w)], pos, fr), INV, "GPU")
    _raises(lambda: f([], pos, fr), INV, "parts")
    _raises(lambda: f([(q, w)], pos[:2], fr), INV, "positions")
    _raises(lambda: f([(q, w)], pos.int(), fr), INV, "positions")
    _raises(lambda: f([(q, w)], pos, fr.float()), INV, "freqs")
    _raises(lambda: f([(q, w)], pos, None), INV, "together")
    _raises(lambda: f([(q, w)], pos, torch.zeros(33, dtype=torch.float64)), INV, "rotated")
    _raises(lambda: f([(q, w[:8])], pos, fr), INV, "weight")
    _raises(lambda: f([(q, w), (k[:2], w)], pos, fr), INV, "part 1")
    _raises(lambda: f([(q, w), (k.float(), w)], pos, fr), INV, "part 1")
    _raises(lambda: f([(q, w)], pos, fr, outs=[k]), INV, "out")
    _raises(lambda: f([(q, w)], pos, fr, outs=[q, k]), INV, "output per part")
    _raises(lambda: f([(q[0], w)], pos, fr), INV, "heads")


def test_binding_refuses_wrong_qkv():
    x = torch.zeros(3, 64, dtype=BF)
    b = lambda o: (torch.zeros(o, dtype=BF), torch.zeros(o, 64, dtype=BF), None, None)   # noqa: E731
    e = lambda o: (torch.zeros(o, 64, dtype=tb.E4M3), torch.zeros(-(-o // 128), 1))   # noqa: E731
    pos, fr = torch.arange(3), torch.zeros(32, dtype=torch.float64)
    f = tb.qkv_forward
    _raises(lambda: f(x, b(256), b(64), b(64), 64, pos, fr), INV, "GPU")
    _raises(lambda: f(x, b(256), e(64), b(64), 64, pos, fr), INV, "all")
    _raises(lambda: f(x, b(256), b(96), b(64), 64, pos, fr), INV, "k:")
    _raises(lambda: f(x, e(250), e(64), e(64), 64, pos, fr), INV, "q:")
    _raises(lambda: f(x, e(256), e(64), e(64), 64, pos[:1], fr), INV, "positions")
    _raises(lambda: f(x, e(256), e(64), e(64), 64, pos, fr, q_weight=torch.zeros(32, dtype=BF)), INV, "head weight")
