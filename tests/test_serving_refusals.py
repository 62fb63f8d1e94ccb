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
