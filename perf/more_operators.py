"""Workloads of the operators around the 8-bit integer projections: the row quantiser, the product with a scale per
token and channel, the norms before and after a block with its gate and residual scale, and the position rotation over
several axes.

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
INT8_MAX = 127.0
LEAST = 2.0 ** -100  # fp32 scales: rows and blocks without a larger entry are scaled as if it were one
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------------------------------


def _rows(m, n, dtype, **more):
    return dict(op="rows", m=m, inp=n, dtype=dtype, **more)


def _product(m, out, n, dtype, given, **more):
    """given: x comes in 8 bits with its scales; dtype: of the result, and of an x that does not."""
    return dict(op="product", m=m, out=out, inp=n, dtype=dtype, given=given, **more)


def _norm(m, n, dtype, stream, post, gate, scale, z, **more):
    """stream: type of the residual; gate: none, channel, group (rows of a sequence share a row) or row; z: wide, int8,
    or e4m3 with scales of that type."""
    return dict(op="norm", m=m, n=n, dtype=dtype, stream=stream, post=post, gate=gate, scale=scale, z=z, **more)


def _heads(tokens, q, k, dim, sizes, pairs, cyclic, norm, dtype, **more):
    """sizes: rotated pairs of each axis, as text; cyclic: the axes take pairs in turn."""
    return dict(op="heads", tokens=tokens, q=q, k=k, dim=dim, sizes=sizes, pairs=pairs, cyclic=cyclic, norm=norm,
                dtype=dtype, **more)


def listed():
    return [
        # A down projection of the 60-layer stack, quantised when it is loaded.
        _rows(5376, 21504, "bf16", name="rows 5376 x 21504"),
        # Activations of a ragged decode batch of the 26-layer stack, quantised once for several projections.
        _rows(61, 1152, "f32", name="rows 61 x 1152"),
        # One token through the stacked q, k, v weight of a 26-layer stack's layer: the smallest call, latency counts.
        _product(1, 1536, 1152, "bf16", False, name="product 1 x 1536 x 1152"),
        # One token through the 60-layer stack's down projection: the weight stream counts.
        _product(1, 5376, 21504, "bf16", False, name="product 1 x 5376 x 21504"),
        # A decode batch of 16 through the 60-layer stack's gate projection, behind a norm that wrote 8 bits.
        _product(16, 21504, 5376, "bf16", True, name="product 16 x 21504 x 5376"),
        # A ragged prompt through the 26-layer stack's down projection, in fp32.
        _product(777, 1152, 6912, "f32", False, name="product 777 x 1152 x 6912"),
        # A long prefill through the 60-layer stack's gate projection: the matrix rate counts.
        _product(4096, 21504, 5376, "bf16", False, name="product 4096 x 21504 x 5376"),
        # One decode token of the 26-layer stack between two blocks: latency counts.
        _norm(1, 1152, "bf16", "bf16", True, "none", 1.0, "wide", name="norm 1 x 1152"),
        # A prefill of the 60-layer stack between two blocks, with a gate per channel: the traffic counts.
        _norm(4096, 5376, "bf16", "bf16", True, "channel", 1.0, "wide", name="norm 4096 x 5376"),
        # A ragged prompt with its residual in fp32, gated by sequence, into the 8-bit blocks of the next projections.
        _norm(1022, 5376, "bf16", "f32", False, "group", 0.7, "e8m0", name="norm 1022 x 5376 to 8 bits"),
        # A prefill of text, images and video in the 60-layer stack: time, height and width.
        _heads(4096, 32, 8, 256, "32,48,48", "half", False, True, "bf16", name="heads 4096 x (32+8) x 256"),
        # The patches of an image encoder: height and width, each in its own half of a head, no norm.
        _heads(1009, 16, 16, 72, "18,18", "axis", False, False, "f32", name="heads 1009 x (16+16) x 72"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rows", "product", "product", "norm", "heads"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "rows":
        m, n = _log(rng, 1, 21504), 8 * _log(rng, 8, 21504 // 8)
        while m * n > 21504 * 5376:
            m = max(1, m // 2)
        return _rows(m, n, dtype)
    if op == "product":
        m = _log(rng, 1, 4096)
        out = _log(rng, 100, 21504)
        n = 16 * _log(rng, 8, 21504 // 16)
        while m * out * n > 4096 * 21504 * 5376 or out * n > 21504 * 5376:
            out, n = max(100, out // 2), max(128, n // 32 * 16)
        return _product(m, out, n, dtype, rng.choice((False, True)))
    if op == "norm":
        z = rng.choice(("wide", "wide", "int8", "f32", "e8m0"))
        n = _log(rng, 64, 8192)
        return _norm(_log(rng, 1, 4096), n if z == "wide" else (n + 7) // 8 * 8, dtype, rng.choice(("bf16", "f32")),
                     rng.choice((False, True)), rng.choice(("none", "channel", "group", "row")),
                     rng.choice((1.0, 0.5, 1.25)), z)
    axes, pairs = rng.randint(2, 4), rng.choice(("half", "interleaved", "axis"))
    sizes = [rng.randint(1, 32) for _ in range(axes)]
    dim = 2 * sum(sizes) + 2 * rng.randint(0, 16)
    return _heads(_log(rng, 1, 4096), rng.randint(1, 32), rng.randint(1, 8), dim, ",".join(map(str, sizes)), pairs,
                  pairs != "axis" and rng.choice((False, True)), rng.choice((False, True)), dtype)


def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    es = _size(case["dtype"])
    if case["op"] == "rows":
        m, n = case["m"], case["inp"]
        return {"bytes": m * n * (es + 1) + 4 * m, "flops": 3 * m * n}
    if case["op"] == "product":
        m, out, n = case["m"], case["out"], case["inp"]
        x = m * n + 4 * m if case["given"] else m * n * es
        return {"bytes": x + out * n + 4 * out + m * out * es, "flops": 2 * m * out * n}
    if case["op"] == "norm":
        m, n, hs = case["m"], case["n"], _size(case["stream"])
        held = m * n * es if case["z"] == "wide" else m * n + 4 * m if case["z"] == "int8" else \
            m * n + m * -(-n // BLOCK) * (4 if case["z"] == "f32" else 1)
        return {"bytes": m * n * (2 * hs + es) + held, "flops": 12 * m * n}
    n = case["tokens"] * (case["q"] + case["k"]) * case["dim"]
    return {"bytes": 2 * n * es + 8 * case["tokens"] * len(case["sizes"].split(",")), "flops": 9 * n}


def _axes(case):
    """The axis of each rotated pair."""
    turns = [(i, a) for a, s in enumerate(case["sizes"].split(",")) for i in range(int(s))]
    return tuple(a for _, a in (sorted(turns) if case["cyclic"] else turns))


# --------------------------------------------------------------------------------------------------------------------
# Plain forms: elementary operations in fp32
# --------------------------------------------------------------------------------------------------------------------


def _plain_rows(x):
    """x [m, n] as int8 with one scale per row.  A quotient with a constant is the product with its reciprocal."""
    xf = x.float()
    amax = xf.abs().amax(1).clamp_min(LEAST)
    q = (xf * (INT8_MAX * (1.0 / amax))[:, None]).round()
    return q.to(torch.int8), amax * (1.0 / INT8_MAX)


def _plain_product(x, xs, wq, ws, dtype):
    if xs is None:
        x, xs = _plain_rows(x)
    return ((x.float() @ wq.float().t()) * (xs[:, None] * ws[None, :])).to(dtype)


def _plain_blocks(z, kind):
    """z [m, n] as e4m3 with one scale per row and 128 columns."""
    m, n = z.shape
    kb = -(-n // BLOCK)
    padded = torch.nn.functional.pad(z, (0, kb * BLOCK - n)).view(m, kb, BLOCK)
    amax = padded.abs().amax(2)
    if kind == "e8m0":
        frac, e = torch.frexp(amax / E4M3_MAX)
        e = torch.where(frac == 0.5, e - 1, e).clamp(-127, 127)  # the least power of two that is >= amax / 448
        stored, by = (e + 127).to(torch.uint8).view(E8M0), torch.ldexp(torch.ones_like(amax), -e)
    else:
        amax = amax.clamp_min(LEAST)
        stored, by = amax * (1.0 / E4M3_MAX), E4M3_MAX * (1.0 / amax)
    return (padded * by[:, :, None]).view(m, kb * BLOCK)[:, :n].to(E4M3), stored


def _plain_normed(x, weight):
    return x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * (weight.float() + 1.0)


def _plain_norm(h, y, post_weight, gate, weight, scale, z):
    a = y.float()
    if post_weight is not None:
        a = _plain_normed(a, post_weight)
    if gate is not None:
        g = gate.float().reshape(-1, gate.shape[-1])
        a = a * g.repeat_interleave(h.shape[0] // g.shape[0], 0)
    hn = h.float() * scale + a
    zf = _plain_normed(hn, weight)
    held = zf.to(y.dtype) if z == "wide" else _plain_rows(zf) if z == "int8" else _plain_blocks(zf, z)
    return hn.to(h.dtype), held


def _plain_heads(x, weight, positions, axes, freqs, size, pairs):
    z = x.float()
    if weight is not None:
        z = z * torch.rsqrt((z * z).mean(2, keepdim=True) + EPS) * (weight.float() + 1.0)
    angle = positions[axes].double().t() * freqs[None, :]  # far positions need more than 32 bits
    c, s = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    half = freqs.numel()
    p = torch.arange(half, device=x.device)
    if pairs == "half":
        i, j = p, p + half
    elif pairs == "interleaved":
        i, j = 2 * p, 2 * p + 1
    else:  # an axis's pairs lie in its own span: pair j of n and its mate n further on
        start = torch.cumsum(size, 0) - size
        i = p + start[axes]
        j = i + size[axes]
    a, b = z[:, :, i], z[:, :, j]
    out = z.clone()
    out[:, :, i] = a * c - b * s
    out[:, :, j] = b * c + a * s
    return out.to(x.dtype)


# --------------------------------------------------------------------------------------------------------------------
# Inputs and passes
# --------------------------------------------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "rows":
        # Rows and channels that differ in size.
        m, n = case["m"], case["inp"]
        return {"case": case, "x": (normal(m, n) * torch.exp(0.5 * normal(n)) * torch.exp(0.3 * normal(m, 1))).to(dtype)}
    if case["op"] == "product":
        m, out, n = case["m"], case["out"], case["inp"]
        # Activations whose channels differ in size, weights of a trained layer's size quantised at load time.
        x, xs = (normal(m, n) * torch.exp(0.5 * normal(n))).to(dtype), None
        if case["given"]:
            x, xs = _plain_rows(x)
        wq, ws = _plain_rows(normal(out, n) * (0.02 * torch.exp(0.2 * normal(out)))[:, None])
        return {"case": case, "x": x, "xs": xs, "wq": wq, "ws": ws}
    if case["op"] == "norm":
        m, n = case["m"], case["n"]
        # A residual stream that has grown, a few of its channels large; a block's output; weights held around one.
        h = (normal(m, n) * 3 * torch.exp(0.7 * normal(n))).to(DTYPES[case["stream"]])
        y = (normal(m, n) * 0.5).to(dtype)
        groups = max(d for d in range(1, 9) if m % d == 0)  # sequences of one length
        gate = {"none": None, "channel": (n,), "group": (groups, n), "row": (m, 1)}[case["gate"]]
        return {"case": case, "h": h, "y": y, "gate": None if gate is None else (1 + 0.3 * normal(*gate)).to(dtype),
                "post": (0.2 * normal(n)).to(dtype) if case["post"] else None, "weight": (0.2 * normal(n)).to(dtype)}
    t, hq, hk, d = case["tokens"], case["q"], case["k"], case["dim"]
    q, k = normal(t, hq, d).to(dtype), normal(t, hk, d).to(dtype)
    wq = (0.1 * normal(d)).to(dtype) if case["norm"] else None
    wk = (0.1 * normal(d)).to(dtype) if case["norm"] else None
    # Patches of a clip 32 wide and 24 high behind some text: each axis counts on its own.
    at = torch.arange(t, device="cuda")
    grid = [at // 768 + 4000, at // 32 % 24 + 4000, at % 32 + 4000, at + 100000]
    axes = _axes(case)
    half = len(axes)
    freqs = 1e4 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    return {"case": case, "q": q, "k": k, "wq": wq, "wk": wk, "positions": torch.stack(grid[:max(axes) + 1]),
            "axes": axes, "axis_of": torch.tensor(axes, device="cuda"), "freqs": freqs,
            "size": torch.bincount(torch.tensor(axes, device="cuda"))}


def run(state):
    case = state["case"]
    if own:
        from rank_factored_linear_amd import binding as tb

        if case["op"] == "rows":
            return tb.quantize_rows_int8(state["x"])
        if case["op"] == "product":
            return tb.dense_forward_int8(state["x"], state["wq"], state["ws"], x_scale=state["xs"],
                                         out_dtype=DTYPES[case["dtype"]])
        if case["op"] == "norm":
            z = case["z"]
            held = None if z == "wide" else torch.int8 if z == "int8" else E4M3
            h, got = tb.residual_norm(state["h"], state["y"], state["weight"], post_norm=case["post"],
                                      post_weight=state["post"], gate=state["gate"], residual_scale=case["scale"],
                                      eps=EPS, weight_offset=1.0, out_dtype=held,
                                      scale_dtype=E8M0 if z == "e8m0" else torch.float32)
        else:
            return tb.head_norm_rotate([(state["q"], state["wq"]), (state["k"], state["wk"])], state["positions"],
                                       state["freqs"], eps=EPS, weight_offset=1.0,
                                       interleaved=case["pairs"] == "interleaved", axes=state["axes"],
                                       axis_halves=case["pairs"] == "axis", norm=case["norm"])
    elif case["op"] == "rows":
        return _plain_rows(state["x"])
    elif case["op"] == "product":
        return _plain_product(state["x"], state["xs"], state["wq"], state["ws"], DTYPES[case["dtype"]])
    elif case["op"] == "norm":
        h, got = _plain_norm(state["h"], state["y"], state["post"], state["gate"], state["weight"], case["scale"],
                             case["z"])
    else:
        more = (state["positions"], state["axis_of"], state["freqs"], state["size"], case["pairs"])
        return [_plain_heads(state["q"], state["wq"], *more), _plain_heads(state["k"], state["wk"], *more)]
    if case["z"] == "int8":  # as the values it stands for: sums in another order may round to the next whole number
        got = (got[0].float() * got[1][:, None]).to(torch.bfloat16)
    return [h, got]


# --------------------------------------------------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# --------------------------------------------------------------------------------------------------------------------


def _nearest_e4m3(v):
    """The nearest of the numbers k * 2^(e - 3), e >= -6, to each fp64 value (ties to even k)."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -30))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _exact_rows(a):
    """(whole numbers, scales) of fp32 values in fp64: the factor and its products are fp32 numbers by definition."""
    top = a.abs().max(1).values.clamp(min=LEAST).float()
    by = (127.0 * top.reciprocal())[:, None]
    return torch.round((a.float() * by).double()), (top * (1.0 / 127.0)).double()


def _exact_normed(x, w):
    return x / torch.sqrt((x ** 2).sum(1, keepdim=True) / x.shape[1] + EPS) * (1 + w.double())


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rows":
        q, s = _exact_rows(st["x"].double())
        return q.to(torch.int8), s
    if case["op"] == "product":
        x, xs = (st["x"].double(), st["xs"].double()) if case["given"] else _exact_rows(st["x"].double())
        y = torch.zeros(case["m"], case["out"], dtype=torch.float64, device="cuda")
        for at in range(0, case["inp"], 1024):  # 1024 products of 127 x 127 add up to less than 2^24: exact in any order
            y += torch.mm(x[:, at:at + 1024].float(), st["wq"][:, at:at + 1024].float().t())
        return y.mul_(xs[:, None]).mul_(st["ws"].double()[None, :])
    if case["op"] == "norm":
        a = st["y"].double()
        if case["post"]:
            a = _exact_normed(a, st["post"])
        m, n = a.shape
        if st["gate"] is not None:
            g = st["gate"].double()
            g = g.view(1, n) if g.dim() == 1 else g
            a = (a.view(g.shape[0], -1, n) * g[:, None, :]).view(m, n)
        h = a + case["scale"] * st["h"].double()
        z = _exact_normed(h, st["weight"])
        if case["z"] == "wide":
            return [h, z]
        if case["z"] == "int8":
            top = z.abs().max(1, keepdim=True).values
            return [h, torch.round(z / top * 127) * (top / 127)]
        kb = -(-n // BLOCK)
        big = torch.zeros(m, kb * BLOCK, dtype=torch.float64, device="cuda")
        big[:, :n] = z
        big = big.view(m, kb, BLOCK)
        s = big.abs().max(2).values / 448
        if case["z"] == "e8m0":
            s = torch.exp2(torch.ceil(torch.log2(s.clamp_min(2.0 ** -127))))
        return [h, [_nearest_e4m3(big / s[:, :, None]).view(m, kb * BLOCK)[:, :n].contiguous(), s]]
    sizes, got = [int(s) for s in case["sizes"].split(",")], []
    half = sum(sizes)
    place = {"half": lambda p: (p, p + half), "interleaved": lambda p: (2 * p, 2 * p + 1)}.get(case["pairs"])
    if place is None:
        start = [sum(sizes[:a]) for a in range(len(sizes))]
        place = lambda p: (start[st["axes"][p]] + p, start[st["axes"][p]] + p + sizes[st["axes"][p]])  # noqa: E731
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        z = x.double()
        if w is not None:
            z = z / torch.sqrt((z ** 2).sum(2, keepdim=True) / case["dim"] + EPS) * (1 + w.double())
        out = z.clone()
        for p, axis in enumerate(st["axes"]):
            turn = (st["positions"][axis].double() * st["freqs"][p])[:, None]
            i, j = place(p)
            out[:, :, i] = z[:, :, i] * torch.cos(turn) - z[:, :, j] * torch.sin(turn)
            out[:, :, j] = z[:, :, j] * torch.cos(turn) + z[:, :, i] * torch.sin(turn)
        got.append(out)
    return got
