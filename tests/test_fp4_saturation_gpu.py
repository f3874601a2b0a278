"""Quantisation with a matrix's scale far too small for the elements: what is above the grid becomes its
largest number of the same sign, also where another element of the block lies on a border."""
import pytest
import torch

import combine_topk_ids_expert_gb300 as ep
from test_fp4_gpu import assert_quantized, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("g", [2.0 ** -60, 2.0 ** -40, 0.9 * 2.0 ** -59])
def test_elements_above_the_grid_beside_one_on_a_border(g):
    ts = torch.tensor([g], device="cuda")
    top = 448 * float(ts)          # the blocks' scale, saturated
    x = torch.zeros((8, 256), device="cuda")
    x[:, 0::16] = 2.5 * top        # on (or, rounded to bf16, near) the border of 2 and 3
    x[:, 1::16] = 0.75 * top
    # From just above the grid to the largest bf16: quotients that overflow, and some that do not.
    powers = torch.arange(-55, 128, device="cuda").double()
    far = torch.exp2(powers) * 1.9921875
    far = far[far > 8 * top].float()
    pick = torch.randint(0, len(far), (8, 16, 12), device="cuda", generator=gen(1))
    sign = 1.0 - 2.0 * torch.randint(0, 2, pick.shape, device="cuda", generator=gen(2))
    x.view(8, 16, 16)[:, :, 2:14] = far[pick] * sign
    x[:, 14::16] = -far[-1]
    x[:, 15::16] = far[-1]
    x = x.bfloat16()
    assert torch.isfinite(x).all()
    q = ep.quantize_fp4(x, "nv", ts)
    assert_quantized(q, x, float(ts))
    v = q.dequantize(torch.float32).view(8, 16, 16)
    assert (v[:, :, 14] == -v[:, :, 15]).all() and (v[:, :, 15] > 0).all()
