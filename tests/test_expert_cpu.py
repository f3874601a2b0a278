"""The experts' operators without a GPU: argument checks that need none."""
import ctypes as C

import pytest
import torch

import combine_topk_ids_expert_gb300 as ep
from combine_topk_ids_expert_gb300 import _abi
from combine_topk_ids_expert_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_w4_shapes_and_types():
    w = ep.W4(codes(2, 8, 64), torch.ones((2, 8, 2)), codes(2, 8, 2))
    assert (w.din, w.rows, w.group) == (128, 8, 64)
    assert ep.W4(codes(2, 8, 64), torch.ones((2, 8, 1), dtype=torch.bfloat16)).group == 128
    with pytest.raises(TypeError, match="codes"):
        ep.W4(torch.zeros((2, 8, 64)), torch.ones((2, 8, 2)))
    with pytest.raises(TypeError, match="scales"):
        ep.W4(codes(2, 8, 64), torch.ones((2, 8, 2), dtype=torch.float64))
    for scales in ((2, 8, 3), (2, 7, 2), (2, 8, 0), (16, 2)):
        with pytest.raises(ValueError, match="fit"):
            ep.W4(codes(2, 8, 64), torch.ones(scales))
    with pytest.raises(ValueError, match="zeros"):
        ep.W4(codes(2, 8, 64), torch.ones((2, 8, 2)), codes(2, 8, 1))
    with pytest.raises(TypeError, match="zeros"):
        ep.W4(codes(2, 8, 64), torch.ones((2, 8, 2)), torch.zeros((2, 8, 2)))
    with pytest.raises(AttributeError):
        w.codes = codes(2, 8, 64)


def test_w4_on_the_host_is_refused():
    w = ep.W4(codes(2, 8, 64), torch.ones((2, 8, 2)))
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ep.ep_expert_gemv_w4(None, x, w, 128, 8, x, stream=0)


def test_no_buffer_is_an_argument_error():
    L = _abi.lib()
    w = _abi.EpW4()
    assert L.ep_expert_glu(None, None, None, 64, 128, 0, None, None, None) == _abi.EP_ERR_INVALID_ARG
    assert L.ep_expert_glu_backward(None, None, None, None, 128, 128, 0, None,
                                    None) == _abi.EP_ERR_INVALID_ARG
    assert L.ep_expert_gemm_backward(None, None, None, None, 64, 128, None, None, 0, 0,
                                     None) == _abi.EP_ERR_INVALID_ARG
    assert L.ep_expert_gemv_w4(None, None, C.byref(w), 64, 8, None, None) == _abi.EP_ERR_INVALID_ARG
    assert L.ep_expert_glu_w4(None, None, C.byref(w), 64, 8, 0, None, None) == _abi.EP_ERR_INVALID_ARG
    assert L.ep_expert_glu_w4(None, None, C.byref(w), 64, 8, 5, None, None) == _abi.EP_ERR_INVALID_ARG
