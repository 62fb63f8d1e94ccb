"""Head norms and rotation where inputs or weights are not finite, against the float64 oracle."""

import numpy as np
import pytest
import torch

from oracle import serving as o
from parity_util import exact
from test_gpu_heads import check, frequencies, randn

pytestmark = pytest.mark.gpu

tb = pytest.importorskip("rank_factored_linear_amd.binding")
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32

# Chunks of 16 bytes, of two elements and of one; rotated in part, in an odd number of pairs, or not at all.
SIZES = [(64, 32), (64, 0), (80, 16), (256, 128), (130, 66), (62, 6), (15, 4), (33, 0)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("d,rot", SIZES)
def test_an_element_that_is_not_rotated_reaches_no_other(d, rot, bad, dtype, interleaved):
    """A weight or an infinite x element that is not finite touches its own element and, where that is rotated, its
    partner: the elements behind rot_dim are y = z."""
    print(d, rot, bad, dtype, interleaved, flush=True)
    pos, fr = torch.arange(3, 6, device=DEV), frequencies(rot)
    for at in sorted({0, 1, rot // 2, max(rot - 1, 0), min(rot, d - 1), min(rot + 1, d - 1), d - 2, d - 1}):
        x, w = randn((3, 2, d), 1, 1.0, dtype), randn((d,), 2, 1.0, dtype)
        w[at] = bad
        y, = tb.head_norm_rotate([(x, w)], pos, fr, interleaved=interleaved)
        with np.errstate(all="ignore"):
            want = o.head_norm_rotate(exact(x), exact(w), pos.cpu().numpy(), fr.cpu().numpy(), 1e-6, 0.0, interleaved)
        assert np.array_equal(np.isfinite(exact(y)), np.isfinite(want)), at
        w[at] = 1
        if bad == bad:
            x[1, 1, at] = bad      # its head's other elements are zero
            y, = tb.head_norm_rotate([(x, w)], pos, fr, interleaved=interleaved)
            with np.errstate(all="ignore"):
                want = o.head_norm_rotate(exact(x), exact(w), pos.cpu().numpy(), fr.cpu().numpy(), 1e-6, 0.0, interleaved)
            assert np.array_equal(np.isnan(exact(y)), np.isnan(want)), at
            assert (exact(y)[1, 1][np.isfinite(want[1, 1])] == 0).all()
            keep = torch.tensor([0, 2], device=DEV)
            check(y[keep], x[keep], w, pos[keep], fr, 1e-6, 0.0, interleaved)
