"""Workloads of the serving operators that go with the projections: the 8-bit block-scaled product, the rebuild of a
bundle into 8-bit blocks, and the head norms with the position rotation.

Each case runs either in plain torch (``own`` false) or through the library's entry points (``own`` true), on the
same inputs.  Sizes are those of the 26-layer stack (hidden 1152, MLP 6912) and of the 60-layer stack (hidden 5376,
MLP 21504), and ragged ones.
"""

import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
BLOCK = 128
E4M3_MAX = 448.0
LEAST = 2.0 ** -100  # fp32 scales: blocks without a larger entry are scaled as if it were one
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SCALES = {"f32": torch.float32, "e8m0": E8M0}


# --------------------------------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------------------------------


def _product(m, out, n, dtype, scale, **more):
    return dict(op="product", m=m, out=out, inp=n, dtype=dtype, scale=scale, **more)


def _rebuild(out, n, rank, dtype, scale, **more):
    return dict(op="rebuild", out=out, inp=n, rank=rank, dtype=dtype, scale=scale, **more)


def _heads(tokens, q, k, dim, rot, dtype, first, pairs, offset, packed, **more):
    return dict(op="heads", tokens=tokens, q=q, k=k, dim=dim, rot=rot, dtype=dtype, first=first, pairs=pairs,
                offset=offset, packed=packed, **more)


def listed():
    return [
        # One token through the stacked q, k, v weight of a 26-layer stack's layer: the smallest call, latency counts.
        _product(1, 1536, 1152, "bf16", "e8m0", name="product 1 x 1536 x 1152"),
        # One token through the 60-layer stack's down projection: the weight stream counts.
        _product(1, 5376, 21504, "bf16", "f32", name="product 1 x 5376 x 21504"),
        # A decode batch of 16 through the 60-layer stack's gate projection.
        _product(16, 21504, 5376, "bf16", "e8m0", name="product 16 x 21504 x 5376"),
        # A ragged decode batch through the 26-layer stack's gate projection.
        _product(61, 6912, 1152, "bf16", "f32", name="product 61 x 6912 x 1152"),
        # A ragged prompt through the 26-layer stack's down projection, in fp32.
        _product(777, 1152, 6912, "f32", "e8m0", name="product 777 x 1152 x 6912"),
        # A long prefill through the 60-layer stack's gate and o projections: the matrix rate counts.
        _product(4096, 21504, 5376, "bf16", "f32", name="product 4096 x 21504 x 5376"),
        _product(4096, 5376, 8192, "bf16", "e8m0", name="product 4096 x 5376 x 8192"),
        # Rebuilding a bundle at load time: a q projection of the 26-layer stack, an up projection of the 60-layer one.
        _rebuild(1024, 1152, 128, "bf16", "e8m0", name="rebuild 1024 x 1152 r128"),
        _rebuild(21504, 5376, 256, "bf16", "f32", name="rebuild 21504 x 5376 r256"),
        # One decode token of the 26-layer stack (4 query heads, 1 key head) far into a context.
        _heads(1, 4, 1, 256, 256, "bf16", 131071, "half", 1.0, False, name="heads 1 x (4+1) x 256"),
        # A prefill of the 60-layer stack, q and k as views of packed q, k, v rows.
        _heads(4096, 32, 8, 256, 256, "bf16", 0, "half", 1.0, True, name="heads 4096 x (32+8) x 256"),
        # fp32 heads of an odd size, rotated in part and in interleaved pairs.
        _heads(1001, 5, 1, 80, 32, "f32", 777, "interleaved", 0.0, False, name="heads 1001 x (5+1) x 80"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("product", "product", "rebuild", "heads"))
    scale = rng.choice(("f32", "e8m0"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "product":
        m = _log(rng, 1, 4096)
        out = _log(rng, 100, 21504)
        n = 16 * _log(rng, 8, 21504 // 16)
        while m * out * n > 4096 * 21504 * 5376 or out * n > 21504 * 5376:
            out, n = max(100, out // 2), max(128, n // 32 * 16)
        return _product(m, out, n, dtype, scale)
    if op == "rebuild":
        out, n = _log(rng, 100, 21504), 8 * _log(rng, 16, 21504 // 8)
        while out * n > 21504 * 5376:
            out, n = max(100, out // 2), max(128, n // 16 * 8)
        return _rebuild(out, n, rng.choice((0, 8, 40, 64, 128, 136, 256)), dtype, scale)
    dim = 2 * rng.randint(32, 128)
    return _heads(_log(rng, 1, 4096), rng.randint(1, 32), rng.randint(1, 8), dim, 2 * rng.randint(1, dim // 2), dtype,
                  rng.randint(0, 1 << 20), rng.choice(("half", "interleaved")), rng.choice((0.0, 1.0)),
                  rng.choice((False, True)))


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "heads":
        n = case["tokens"] * (case["q"] + case["k"]) * case["dim"]
        return {"bytes": 2 * n * es + 8 * case["tokens"], "flops": 9 * n}
    out, n = case["out"], case["inp"]
    ss = 4 if case["scale"] == "f32" else 1
    blocks = -(-out // BLOCK) * -(-n // BLOCK)
    if case["op"] == "rebuild":
        r = case["rank"]
        return {"bytes": out * n * (es + 1) + (out + (out + n) * r) * es + blocks * ss, "flops": 2 * out * n * (r + 1)}
    m = case["m"]
    return {"bytes": m * n * es + out * n + blocks * ss + m * out * es, "flops": 2 * m * out * n}


# --------------------------------------------------------------------------------------------------------------------
# Plain forms: elementary operations in fp32
# --------------------------------------------------------------------------------------------------------------------


def _scales(amax, scale):
    """(the scale as it is stored, what a value is multiplied by) for blocks of largest magnitude amax."""
    if scale == "e8m0":
        frac, e = torch.frexp(amax / E4M3_MAX)
        e = torch.where(frac == 0.5, e - 1, e).clamp(-127, 127)  # the least power of two that is >= amax / 448
        return (e + 127).to(torch.uint8).view(E8M0), torch.ldexp(torch.ones_like(amax), -e)
    amax = amax.clamp_min(LEAST)
    return amax / E4M3_MAX, E4M3_MAX / amax


def _quantise_rows(x, scale):
    """x [m, n] with one scale per row and 128 columns: (e4m3 [m, n], scales [m, n / 128 rounded up])."""
    m, n = x.shape
    kb = -(-n // BLOCK)
    padded = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - n)).view(m, kb, BLOCK)
    stored, by = _scales(padded.abs().amax(2), scale)
    return (padded * by[:, :, None]).view(m, kb * BLOCK)[:, :n].to(E4M3), stored


def _quantise_blocks(w, scale):
    """w [out, n] with one scale per 128 x 128 block: (e4m3 [out, n], scales [out / 128, n / 128, rounded up])."""
    out, n = w.shape
    ob, kb = -(-out // BLOCK), -(-n // BLOCK)
    padded = torch.nn.functional.pad(w.float(), (0, kb * BLOCK - n, 0, ob * BLOCK - out)).view(ob, BLOCK, kb, BLOCK)
    stored, by = _scales(padded.abs().amax((1, 3)), scale)
    return (padded * by[:, None, :, None]).view(ob * BLOCK, kb * BLOCK)[:out, :n].to(E4M3).contiguous(), stored


def _spread(scale, out, n, rows):
    """Block scales as one fp32 value per entry of an [out, n] matrix."""
    s = scale.float().repeat_interleave(BLOCK, 1)[:, :n]
    return s.repeat_interleave(BLOCK, 0)[:out] if rows else s


def _plain_product(x, wq, ws, scale):
    xq, xs = _quantise_rows(x, scale)
    out, n = wq.shape
    a = xq.float() * _spread(xs, x.shape[0], n, False)
    b = wq.float() * _spread(ws, out, n, True)
    return (a @ b.t()).to(x.dtype)


def _plain_rebuild(s, w0, u, v, scale):
    w = w0.float() * s.float()[:, None]
    if u is not None:
        w = w + u.float() @ v.float().t()
    return _quantise_blocks(w, scale)


def _plain_heads(x, weight, positions, freqs, eps, offset, pairs):
    xf = x.float()
    z = xf * torch.rsqrt((xf * xf).mean(2, keepdim=True) + eps) * (weight.float() + offset)
    angle = positions.double()[:, None] * freqs[None, :]  # far positions need more than 32 bits
    c, s = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    half = freqs.numel()
    if pairs == "half":
        a, b = z[:, :, :half], z[:, :, half:2 * half]
        turned = torch.cat((a * c - b * s, b * c + a * s), 2)
    else:
        a, b = z[:, :, 0:2 * half:2], z[:, :, 1:2 * half:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), 3).flatten(2)
    return torch.cat((turned, z[:, :, 2 * half:]), 2).to(x.dtype)


# --------------------------------------------------------------------------------------------------------------------
# Inputs and passes
# --------------------------------------------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "product":
        m, out, n = case["m"], case["out"], case["inp"]
        # Activations whose channels differ in size, weights of a trained layer's size quantised at load time.
        x = (normal(m, n) * torch.exp(0.7 * normal(n))).to(dtype)
        wq, ws = _quantise_blocks(normal(out, n) * (0.02 * torch.exp(0.2 * normal(out)))[:, None], case["scale"])
        return {"case": case, "x": x, "wq": wq, "ws": ws}
    if case["op"] == "rebuild":
        out, n, r = case["out"], case["inp"], case["rank"]
        u = (0.02 * normal(out, r)).to(dtype) if r else None
        v = (0.05 * normal(n, r)).to(dtype) if r else None
        return {"case": case, "s": (1 + 0.1 * normal(out)).to(dtype), "w0": (0.02 * normal(out, n)).to(dtype), "u": u,
                "v": v}
    t, hq, hk, d = case["tokens"], case["q"], case["k"], case["dim"]
    if case["packed"]:  # rows of q, k, v as one projection writes them
        rows = normal(t, hq + 2 * hk, d).to(dtype)
        q, k = rows[:, :hq], rows[:, hq:hq + hk]
    else:
        q, k = normal(t, hq, d).to(dtype), normal(t, hk, d).to(dtype)
    wq = (1 - case["offset"] + 0.1 * normal(d)).to(dtype)
    wk = (1 - case["offset"] + 0.1 * normal(d)).to(dtype)
    positions = torch.arange(case["first"], case["first"] + t, device="cuda")
    half = case["rot"] // 2
    freqs = 1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    return {"case": case, "q": q, "k": k, "wq": wq, "wk": wk, "positions": positions, "freqs": freqs}


EPS = 1e-6


def run(state):
    case = state["case"]
    if own:
        from rank_factored_linear_amd import binding as tb

        if case["op"] == "product":
            return tb.dense_forward_fp8(state["x"], state["wq"], state["ws"])
        if case["op"] == "rebuild":
            return tb.reconstruct_weight_fp8(state["s"], state["w0"], state["u"], state["v"],
                                             scale_dtype=SCALES[case["scale"]])
        return tb.head_norm_rotate([(state["q"], state["wq"]), (state["k"], state["wk"])], state["positions"],
                                   state["freqs"], eps=EPS, weight_offset=case["offset"],
                                   interleaved=case["pairs"] == "interleaved")
    if case["op"] == "product":
        return _plain_product(state["x"], state["wq"], state["ws"], case["scale"])
    if case["op"] == "rebuild":
        return _plain_rebuild(state["s"], state["w0"], state["u"], state["v"], case["scale"])
    more = (state["positions"], state["freqs"], EPS, case["offset"], case["pairs"])
    return [_plain_heads(state["q"], state["wq"], *more), _plain_heads(state["k"], state["wk"], *more)]


# --------------------------------------------------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# --------------------------------------------------------------------------------------------------------------------


def _nearest_e4m3(v):
    """The nearest of the numbers k * 2^(e - 3), e >= -6, to each fp64 value (ties to even k)."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -30))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _exact_blocks(a, rows, scale):
    """(values held, scales) of a [m, n] matrix in blocks of `rows` rows and 128 columns, in fp64.  With fp32 scales the
    factor 448 / amax and its products are fp32 numbers by definition; with powers of two nothing is rounded."""
    m, n = a.shape
    mb, kb = -(-m // rows), -(-n // BLOCK)
    big = torch.zeros(mb * rows, kb * BLOCK, dtype=torch.float64, device=a.device)
    big[:m, :n] = a
    big = big.reshape(mb, rows, kb, BLOCK).transpose(1, 2)
    top = big.abs().flatten(2).max(2).values
    if scale == "e8m0":
        s = torch.exp2(torch.ceil(torch.log2((top / 448).clamp_min(2.0 ** -127))))
        held = _nearest_e4m3(big / s[:, :, None, None])
    else:
        top = top.clamp_min(LEAST).float()
        s = (top / 448).double()
        held = _nearest_e4m3((big.float() * (448 / top)[:, :, None, None]).double())
    whole = held.transpose(1, 2).reshape(mb * rows, kb * BLOCK)[:m, :n]
    return whole, s


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "product":
        held, s = _exact_blocks(st["x"].double(), 1, case["scale"])
        x = held * s.repeat_interleave(BLOCK, 1)[:, :held.shape[1]]
        w = st["wq"].double()
        ws = st["ws"].double()
        for b in range(ws.shape[0]):
            w[b * BLOCK:(b + 1) * BLOCK] *= ws[b].repeat_interleave(BLOCK)[:w.shape[1]]
        return torch.mm(x, w.t().contiguous())
    if case["op"] == "rebuild":
        w = st["s"].double()[:, None] * st["w0"].double()
        if st["u"] is not None:
            w += torch.mm(st["u"].double(), st["v"].double().t().contiguous())
        return _exact_blocks(w, BLOCK, case["scale"])
    half, got = case["rot"] // 2, []
    turns = st["positions"].double()[:, None] * st["freqs"]
    turn = torch.complex(torch.cos(turns), torch.sin(turns))[:, None, :]
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        x = x.double()
        z = x / torch.sqrt((x ** 2).sum(2, keepdim=True) / case["dim"] + EPS) * (w.double() + case["offset"])
        if case["pairs"] == "half":
            p = torch.complex(z[..., :half], z[..., half:2 * half]) * turn
            z[..., :half], z[..., half:2 * half] = p.real, p.imag
        else:
            p = torch.complex(z[..., 0:2 * half:2].contiguous(), z[..., 1:2 * half:2].contiguous()) * turn
            z[..., 0:2 * half:2], z[..., 1:2 * half:2] = p.real, p.imag
        got.append(z)
    return got
