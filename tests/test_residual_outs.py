"""residual_norm with an 8-bit z whose scales are missing from outs: refused as any other mismatch is."""

import pytest
import torch

tb = pytest.importorskip("rank_factored_linear_amd.binding")


@pytest.mark.parametrize("out_dtype", [None, torch.int8, tb.E4M3])
@pytest.mark.parametrize("held", [torch.int8, tb.E4M3])
@pytest.mark.parametrize("scales", [(), (None,)])
def test_an_8_bit_z_without_its_scales(scales, held, out_dtype):
    h, y = torch.zeros(6, 64), torch.zeros(6, 64, dtype=torch.bfloat16)
    with pytest.raises(tb.TBError) as e:
        tb.residual_norm(h, y, out_dtype=out_dtype, outs=(h, (torch.zeros(6, 64).to(held), *scales)))
    assert e.value.status == tb.TB_ERR_INVALID_ARGUMENT
    if out_dtype in (None, held):
        assert "scales" in str(e.value)
