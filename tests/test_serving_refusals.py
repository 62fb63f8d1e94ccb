"""Refusals of the serving calls, on the host: the C ABI with addresses that are never used, and the binding with CPU
tensors, where a check that comes late shows as the refusal of the device instead."""

import ctypes

import pytest
import torch

tb = pytest.importorskip("rank_factored_linear_amd.binding")
lib = tb.lib
FAKE = 0x100000
INV, UNS = tb.TB_ERR_INVALID_ARGUMENT, tb.TB_ERR_UNSUPPORTED
BF = torch.bfloat16


def refused(fn, status, word):
    with pytest.raises(tb.TBError) as e:
        fn()
    assert e.value.status == status, str(e.value)
    assert word in str(e.value), str(e.value)


def blocks(out, n=64, scale=torch.float32):
    return torch.zeros(out, n, dtype=tb.E4M3), torch.zeros(-(-out // 128), -(-n // 128), dtype=scale)


def bundle(out, n=64):
    return torch.zeros(out, dtype=BF), torch.zeros(out, n, dtype=BF), None, None


def test_qkv_checks_every_argument_before_the_first_launch():
    x, f = torch.zeros(3, 64, dtype=BF), tb.qkv_forward

    def call(q=blocks(256), k=blocks(64), v=blocks(64), x=x, dim=64, **more):
        return lambda: f(x, q, k, v, dim, None, None, **more)

    refused(call(), INV, "GPU")                                            # well formed but for the device
    refused(call(k=blocks(64, scale=tb.E8M0)), INV, "k: scales")
    refused(call(v=blocks(64, scale=tb.E8M0)), INV, "v: scales")
    refused(call(q=blocks(256, scale=BF)), UNS, "scales")
    refused(call(k=blocks(64, 80)), INV, "Wq")
    refused(call(v=(blocks(64)[0].view(torch.uint8), blocks(64)[1])), INV, "Wq")
    refused(call(v=(blocks(64)[0], torch.zeros(2, 1))), INV, "w_scale")
    refused(call(x=x.half()), UNS, "float16")
    refused(call(x=x[0]), INV, "x must be")
    n8 = torch.zeros(3, 72, dtype=BF)                                      # what the quantiser takes and the product does not
    refused(call(blocks(256, 72), blocks(64, 72), blocks(64, 72), n8), UNS, "multiple of 16")
    for q, k, v in ((blocks(256), blocks(64), blocks(64)), (bundle(256), bundle(64), bundle(64))):
        refused(call(q, k, v, eps=-1.0), INV, "eps")
        refused(call(q, k, v, eps=float("nan")), INV, "eps")
    for kind in (blocks, bundle):
        refused(call(kind(2080), kind(1040), kind(1040), dim=1040), UNS, "head_dim")
        refused(call(kind(65535), kind(1), kind(1), dim=1), UNS, "heads")


# ---- parts of head_norm_rotate that overlap ------------------------------------------------------------------------

ES = 2   # bf16


def heads_call(parts, tokens=5, dim=64):
    """(status, message) of a call that gets no positions: one whose parts are all right is refused for those."""
    arr = (tb.HeadPart * len(parts))()
    for j, (x, y, h, xt, xh, yt, yh) in enumerate(parts):
        arr[j] = tb.HeadPart(FAKE + ES * x, FAKE + ES * y, None, h, xt, xh, yt, yh)
    status = lib.tb_head_norm_rotate(len(parts), arr, tokens, dim, dim, 0, None, None, 1e-6, 0.0, tb.TB_BF16, None)
    return status, lib.tb_last_error().decode()


def elements(base, heads, ts, hs, tokens, dim):
    return {base + t * ts + h * hs + d for t in range(tokens) for h in range(heads) for d in range(dim)}


FAR = 1 << 20


@pytest.mark.parametrize("parts,fine", [
    # Queries and keys as views of packed rows of 8 heads of 64, in place: interleaved, nothing shared.
    ([(0, 0, 4, 512, 64, 512, 64), (256, 256, 2, 512, 64, 512, 64)], True),
    ([(0, 0, 4, 512, 64, 512, 64), (192, 192, 2, 512, 64, 512, 64)], False),            # one head in both
    ([(0, 0, 4, 512, 64, 512, 64), (256 - 8, FAR, 2, 512, 64, 128, 64)], False),        # reads a piece of what q writes
    ([(0, 0, 8, 512, 64, 512, 64), (512 * 4 + 448, 2 * FAR, 1, 512, 64, 64, 64)], False),   # its last token's last head
    ([(0, 0, 7, 512, 64, 512, 64), (448, 448, 1, 512, 9, 512, 9)], True),               # one head: any head stride
    ([(0, FAR, 4, 256, 64, 256, 64), (2 * FAR, FAR + 32, 4, 256, 64, 256, 64)], False),  # outputs half a head apart
    ([(0, FAR, 4, 256, 64, 256, 64), (2 * FAR, FAR + 4 * 256 + 192, 4, 256, 64, 256, 64)], False),   # first on the last row
    ([(0, FAR, 4, 256, 64, 256, 64), (2 * FAR, FAR + 5 * 256, 4, 256, 64, 256, 64)], True),          # right behind it
    ([(0, 32, 4, 256, 64, 256, 64)], False),                                            # y inside x, not x
    ([(0, 256, 4, 256, 64, 256, 64)], False),                                           # one token on
    ([(0, 256, 4, 512, 64, 512, 64)], True),                                            # the other half of packed rows
    # Head-major caches: two slots of one cache, apart and overlapping by a token.
    ([(0, FAR, 2, 128, 64, 64, 640), (2 * FAR, FAR + 320, 2, 128, 64, 64, 640)], True),
    ([(0, FAR, 2, 128, 64, 64, 640), (2 * FAR, FAR + 256, 2, 128, 64, 64, 640)], False),
    # The same x read twice is no conflict.
    ([(0, FAR, 2, 128, 64, 128, 64), (0, 2 * FAR, 2, 128, 64, 128, 64)], True),
    # A part without heads has no rows.
    ([(0, 0, 0, 512, 64, 512, 64), (0, 0, 4, 512, 64, 512, 64)], True),
])
def test_parts_that_overlap_anywhere_are_refused(parts, fine):
    status, message = heads_call(parts)
    assert status == INV
    assert message.startswith("positions") if fine else "overlaps x" in message or "one writes" in message, message


def test_overlap_is_exact_where_strides_agree():
    """Against sets of elements: packed rows of three heads of 6 in steps of 1 element."""
    dim, tokens = 6, 3
    for ts, hs in ((18, 6), (20, 7), (6, 18), (40, 9)):
        for shift in range(-130, 131):
            for ha, hb in ((1, 1), (2, 1), (1, 2), (2, 2)):
                if tokens * hs > 40 and ts < hs and ha + hb > 2 and hs < tokens * ts:
                    continue   # (rows of one tensor would overlap)
                a, b = elements(500, ha, ts, hs, tokens, dim), elements(500 + shift, hb, ts, hs, tokens, dim)
                if len(a) != ha * tokens * dim or len(b) != hb * tokens * dim:
                    continue
                status, message = heads_call([(FAR, 500, ha, ts, hs, ts, hs), (2 * FAR, 500 + shift, hb, ts, hs, ts, hs)],
                                             tokens, dim)
                assert status == INV
                assert message.startswith("positions") == a.isdisjoint(b), (ts, hs, shift, ha, hb, message)


@pytest.mark.parametrize("m,fits,over", [
    (1, 800_000_000, 806_000_000), (16, 800_000_000, 806_000_000), (17, 530_000_000, 537_000_000),
    (32, 530_000_000, 537_000_000), (33, 400_000_000, 403_000_000), (64, 400_000_000, 403_000_000)])
def test_rows_past_one_launch_are_refused(m, fits, over):
    """A launch of the few-token kernel (512 threads for 96, 64 or 48 rows) holds fewer than 2^32 threads."""
    size = ctypes.c_size_t(0)

    def query(out):
        return lib.tb_dense_forward_fp8_workspace_size(m, out, 16, tb.TB_BF16, tb.TB_BF16, tb.TB_SCALE_F32,
                                                       ctypes.byref(size))

    assert query(over) == UNS
    assert query(fits) != UNS           # (without a GPU the query ends at the device)
    assert lib.tb_dense_forward_fp8(FAKE, None, FAKE, FAKE, FAKE, m, over, 16, tb.TB_BF16, tb.TB_BF16, tb.TB_SCALE_F32,
                                    None, 0, None) == UNS
    # The share of a workgroup on 256 compute units, as the kernel takes it.
    most = 96 if m <= 16 else 64 if m <= 32 else 48
    k = -(-fits // (256 * most))
    rows = -(-fits // (256 * k))
    rows = rows if m <= 16 else (rows + 3) // 4 * 4
    assert -(-fits // rows) * 512 < 1 << 32
