"""qkv_forward at the edges of what it takes."""

import pytest
import torch

from test_gpu_heads import frequencies, randn

pytestmark = pytest.mark.gpu

tb = pytest.importorskip("rank_factored_linear_amd.binding")
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("scale", [F32, tb.E8M0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_tokens(dtype, scale):
    """An empty batch through 8-bit weights: empty heads, as from every call under it."""
    x = torch.empty(0, 256, dtype=dtype, device=DEV)
    q, k, v = (tb.quantize_weight(randn((rows, 256), rows, 0.05), scale) for rows in (256, 128, 64))
    pos, fr, w = torch.empty(0, dtype=torch.int64, device=DEV), frequencies(64), randn((64,), 2, 1.0, dtype)
    for angles in ((pos, fr), (None, None)):
        got = tb.qkv_forward(x, q, k, v, 64, *angles, w, w)
        assert [tuple(y.shape) for y in got] == [(0, 4, 64), (0, 2, 64), (0, 1, 64)]
        assert all(y.dtype == dtype and y.is_cuda for y in got)
