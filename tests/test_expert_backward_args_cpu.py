"""expert_gemm_backward says which argument is missing, before anything else is looked at."""
import pytest
import torch

import combine_topk_ids_expert_gb300 as ep


@pytest.mark.parametrize("kw,match", [
    (dict(x_recv=None, weights=None), "weights"),
    (dict(x_recv=torch.zeros((4, 64)), weights=None), "weights"),
    (dict(x_recv=None, weights=torch.zeros((1, 128, 64))), "x_recv"),
    (dict(x_recv=None, weights=None, want_x=False), "x_recv"),
    (dict(x_recv=None, weights=None, want_weights=False), "weights"),
    (dict(x_recv=None, weights=None, want_x=False, want_weights=False), "neither"),
])
def test_missing_arguments_are_named(kw, match):
    buf = ep.Buffer.__new__(ep.Buffer)      # no device: the checks come first
    with pytest.raises(ValueError, match=match):
        buf.expert_gemm_backward(torch.zeros((4, 128)), **kw)
