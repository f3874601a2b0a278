"""Arguments of the 4-bit calls that cannot hold together are refused, before anything else."""
import pytest
import torch

import combine_topk_ids_expert_gb300 as ep


def glu(**kw):
    return ep.Buffer.expert_glu_fp4(None, None, None, **kw)


def test_a_given_h_says_by_itself_how_it_is_held():
    rows = torch.zeros((4, 128), dtype=torch.bfloat16)
    fp4 = ep.FP4(torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((1, 2, 32, 4, 4), dtype=torch.uint8),
                 "nv")
    scale = torch.ones(1)
    for kw in (dict(h=rows, quantize=True), dict(h=rows, h_scale=scale), dict(h=fp4, h_scale=scale),
               dict(h=fp4, quantize=True, h_scale=scale)):
        with pytest.raises(ValueError, match="given h"):
            glu(**kw)


def test_a_scale_of_h_needs_quantisation():
    with pytest.raises(ValueError, match="h_scale needs"):
        glu(h_scale=torch.ones(1))


def test_receive_rows_before_a_dispatch():
    buf = object.__new__(ep.Buffer)          # no GPU needed for what comes first
    buf.R, buf.E, buf.packed, buf._stride = 1, 4, True, None
    rows = ep.FP4(torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((1, 2, 32, 4, 4), dtype=torch.uint8),
                  "nv")
    w = ep.FP4(torch.zeros((4, 128, 64), dtype=torch.uint8),
               torch.zeros((4, 2, 32, 4, 4), dtype=torch.uint8), "nv")
    with pytest.raises(ep.EpError) as e:
        buf.expert_gemm_fp4(rows, w)
    assert e.value.status == ep._abi.EP_ERR_NO_LAYOUT
