"""A step without tokens (num_tokens_per_rank 0, which dispatch accepts) through the experts'
operators: their row operands are tensors of no elements, whose address is NULL. Nothing is
computed, results are empty, and the weights' gradients are zero, or stay as they are when
accumulating."""
import pytest
import torch

import combine_topk_ids_expert_gb300 as ep

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
D, F, E, K = 128, 256, 4, 2


@pytest.fixture(params=["strided", "packed"])
def step(request):
    buf = ep.Buffer(16, D, E, 2, K, dtype=BF16, layout=request.param)
    x = torch.empty((0, D), dtype=BF16, device="cuda")
    ids = torch.empty((0, K), dtype=torch.int32, device="cuda")
    scores = torch.empty((0, K), device="cuda")
    d = buf.dispatch(x, scores, ids)
    yield buf, d.recv_x, scores
    torch.cuda.synchronize()
    assert buf.device_error() == 0
    buf.close()


def ones(*shape, dtype=BF16):
    return torch.ones(shape, dtype=dtype, device="cuda")


def test_gemm(step):
    buf, x, _ = step
    assert buf.expert_gemm(x, ones(E, D, D)).numel() == 0


def test_block_from_dispatch_to_combine_and_back(step):
    buf, x, scores = step
    wgu, wd = ones(E, 2 * F, D), ones(E, D, F)
    y, h, gate_up = buf.expert_ffn(x, wgu, wd, save=True)
    assert y.shape[-1] == D and h.shape[-1] == F and gate_up.shape[-1] == 2 * F
    assert y.numel() == h.numel() == gate_up.numel() == 0
    assert buf.expert_ffn(x, wgu, wd).numel() == 0
    assert buf.combine(y, scores).shape == (0, D)
    grad_y, _ = buf.combine_backward(torch.empty((0, D), dtype=BF16, device="cuda"), y, scores)
    gx, gwgu, gwd = buf.expert_ffn_backward(grad_y, x, wgu, wd, gate_up, h)
    assert gx.numel() == 0 and buf.dispatch_backward(gx, 0)[0].shape == (0, D)
    assert gwgu.shape == wgu.shape and not bool(gwgu.any())
    assert gwd.shape == wd.shape and not bool(gwd.any())


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradients(step, dtype, accumulate):
    buf, x, _ = step
    gu, gd = 7 * ones(E, 2 * F, D, dtype=dtype), 7 * ones(E, D, F, dtype=dtype)
    h, gate_up = x.new_empty(x.shape[:-1] + (F,)), x.new_empty(x.shape[:-1] + (2 * F,))
    got = buf.expert_ffn_backward(x, x, ones(E, 2 * F, D), ones(E, D, F), gate_up, h,
                                  grad_w_gate_up=gu, grad_w_down=gd, accumulate=accumulate)
    assert got[1] is gu and got[2] is gd
    want = 7.0 if accumulate else 0.0
    assert bool((gu == want).all()) and bool((gd == want).all())
    # One at a time: the rows' gradient alone, the weights' alone.
    gx, gw = buf.expert_gemm_backward(x, None, ones(E, D, D), want_weights=False)
    assert gx.numel() == 0 and gw is None
    gw = 5 * ones(E, D, D, dtype=dtype)
    buf.expert_gemm_backward(x, x, None, want_x=False, grad_weights=gw, accumulate=accumulate)
    assert bool((gw == (5.0 if accumulate else 0.0)).all())


def test_four_bit_block(step):
    buf, x, scores = step

    def w4(rows, cols):
        return ep.W4(torch.zeros((E, rows, cols // 2), dtype=torch.uint8, device="cuda"),
                     ones(E, rows, cols // 64))

    assert buf.expert_gemv_w4(x, w4(D, D)).numel() == 0
    assert buf.expert_glu_w4(x, w4(2 * F, D)).numel() == 0
    y = buf.expert_ffn_w4(x, w4(2 * F, D), w4(D, F))
    assert buf.combine(y, scores).shape == (0, D)


def test_missing_weights_are_still_refused(step):
    buf, x, _ = step
    A, H, none = ep._abi, buf.handle, torch.empty((0, D, D), dtype=BF16, device="cuda")

    def status(fn, *args):
        with pytest.raises(ep.EpError) as info:
            fn(*args)
        return info.value.status

    assert status(ep.ep_expert_gemm, H, x, none, D, D, x) == A.EP_ERR_INVALID_ARG
    assert status(ep.ep_expert_glu, H, x, none, D, F, 0, None, x) == A.EP_ERR_INVALID_ARG
    assert status(ep.ep_expert_glu_backward, H, x, none, x, F, D, 0, x) == A.EP_ERR_INVALID_ARG


def test_missing_rows_are_still_refused():
    # With rows, NULL row operands are an error as before.
    buf = ep.Buffer(16, D, E, 2, K, dtype=BF16)
    ids = torch.zeros((4, K), dtype=torch.int32, device="cuda")
    ids[:, 1] = 1
    buf.dispatch_layout(ids, 4)
    A, H, none = ep._abi, buf.handle, torch.empty((0, D), dtype=BF16, device="cuda")
    w4 = ep.W4(torch.zeros((E, D, D // 2), dtype=torch.uint8, device="cuda"), ones(E, D, D // 64))
    for call in (lambda: ep.ep_expert_gemm(H, none, ones(E, D, D), D, D, none),
                 lambda: ep.ep_expert_glu(H, none, ones(E, 2 * F, D), D, F, 0, None, none),
                 lambda: ep.ep_expert_glu_backward(H, none, ones(E, D, F), none, F, D, 0, none),
                 lambda: ep.ep_expert_gemm_backward(H, none, none, ones(E, D, D), D, D, none),
                 lambda: ep.ep_expert_gemm_backward(H, none, none, None, D, D),
                 lambda: ep.ep_expert_gemv_w4(H, none, w4, D, D, none)):
        with pytest.raises(ep.EpError) as info:
            call()
        assert info.value.status == A.EP_ERR_INVALID_ARG
    buf.close()
