"""The router, 4-bit floating point and the layer for a few tokens without a GPU: what their calls
refuse, their sizes, and their structures against the header's."""
import ctypes as C
import os
import shutil
import subprocess

import pytest
import torch

import combine_topk_ids_expert_gb300 as ep
import fp4_util as F4
from combine_topk_ids_expert_gb300 import _abi
from combine_topk_ids_expert_gb300.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_scale_bytes():
    assert ep.ep_fp4_scale_bytes(0, 128, ep.EP_FP4_MX) == 0
    assert ep.ep_fp4_scale_bytes(1, 128, ep.EP_FP4_MX) == 512
    assert ep.ep_fp4_scale_bytes(129, 256, ep.EP_FP4_NV) == 2 * 4 * 512
    for rows, cols, fmt in ((1, 64, 0), (1, 0, 0), (-1, 128, 0), (1, 128, 2), (1, 192, 1)):
        assert ep.ep_fp4_scale_bytes(rows, cols, fmt) == 0


def test_tiles_of_scales():
    s = torch.arange(300 * 8).remainder(251).to(torch.uint8).view(300, 8)
    t = ep.tile_fp4_scales(s)
    assert t.shape == (3, 2, 32, 4, 4) and t.numel() == ep.ep_fp4_scale_bytes(300, 256, ep.EP_FP4_MX)
    assert torch.equal(ep.untile_fp4_scales(t, 300), s)
    assert torch.equal(ep.tile_fp4_scales(s.view(2, 150, 8)), t)     # leading dimensions flattened
    for r, b in [(0, 0), (33, 1), (127, 7), (128, 4), (299, 6)]:
        assert t.flatten()[(r // 128 * 2 + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4] == s[r, b]
    with pytest.raises(TypeError):
        ep.tile_fp4_scales(s.float())
    for bad in (u8(4), u8(4, 6), u8(4, 0)):
        with pytest.raises(ValueError):
            ep.tile_fp4_scales(bad)


def test_fp4_shapes_and_types():
    q = ep.FP4(u8(2, 128, 64), u8(2, 2, 32, 4, 4), "nv", torch.ones(2))
    assert (q.rows, q.cols, q.matrices) == (256, 128, 2)
    assert ep.FP4(u8(5, 64), u8(1, 1, 32, 4, 4), "mx").matrices == 1
    with pytest.raises(ValueError, match="format"):
        ep.FP4(u8(5, 64), u8(1, 1, 32, 4, 4), "e2m1")
    with pytest.raises(TypeError, match="codes"):
        ep.FP4(u8(5, 64).float(), u8(1, 1, 32, 4, 4), "mx")
    with pytest.raises(TypeError, match="scales"):
        ep.FP4(u8(5, 64), u8(1, 1, 32, 4, 4).float(), "mx")
    for codes in (u8(64), u8(5, 32), u8(5, 0)):
        with pytest.raises(ValueError, match="codes"):
            ep.FP4(codes, u8(1, 1, 32, 4, 4), "mx")
    for scales in (u8(1, 2, 32, 4, 4), u8(5, 4), u8(2, 1, 32, 4, 4)):
        with pytest.raises(ValueError, match="scales"):
            ep.FP4(u8(5, 64), scales, "mx")
    with pytest.raises(ValueError, match="tensor_scale"):
        ep.FP4(u8(5, 64), u8(1, 1, 32, 4, 4), "mx", torch.ones(1))
    with pytest.raises(ValueError, match="tensor_scale"):
        ep.FP4(u8(5, 64), u8(1, 2, 32, 4, 4), "nv", torch.ones(2))
    with pytest.raises(TypeError, match="tensor_scale"):
        ep.FP4(u8(5, 64), u8(1, 2, 32, 4, 4), "nv", torch.ones(1, dtype=torch.float64))
    with pytest.raises(AttributeError):
        q.format = "mx"


def test_host_tensors_and_arguments_are_refused():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ep.quantize_fp4(x)
    with pytest.raises(ValueError, match="CUDA"):
        ep.FP4(u8(5, 64), u8(1, 1, 32, 4, 4), "mx").dequantize()
    with pytest.raises(TypeError):
        ep.quantize_fp4(x.float())
    with pytest.raises(ValueError, match="format"):
        ep.quantize_fp4(x, "fp4")
    for bad in (x[0], x[:, :64]):
        with pytest.raises(ValueError, match="cols"):
            ep.quantize_fp4(bad)
    logits = torch.zeros((3, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ep.route(logits, 2)
    with pytest.raises(TypeError):
        ep.route(logits.double(), 2)
    for kw in (dict(topk=0), dict(topk=9), dict(topk=2, score="relu")):
        with pytest.raises(ValueError):
            ep.route(logits, **kw)
    with pytest.raises(ValueError):
        ep.route(logits[0], 1)
    with pytest.raises(TypeError, match="select"):
        ep.route(logits, 2, select=logits.bfloat16())
    with pytest.raises(ValueError, match="select"):
        ep.route(logits, 2, select=logits[:, :4])
    ids = torch.zeros((3, 2), dtype=torch.int32)
    with pytest.raises(TypeError):
        ep.route_backward(torch.zeros((3, 2)), logits, ids.long())
    with pytest.raises(TypeError):
        ep.route_backward(torch.zeros((3, 2), dtype=torch.bfloat16), logits, ids)
    with pytest.raises(ValueError):
        ep.route_backward(torch.zeros((3, 3)), logits, ids)


def test_c_calls_refuse_before_any_gpu_work():
    """Every refusal that needs no buffer: nothing is launched (there is no GPU)."""
    L, p = _abi.lib(), 0x1000
    bad, cap, al = _abi.EP_ERR_INVALID_ARG, _abi.EP_ERR_CAPACITY, _abi.EP_ERR_ALIGNMENT

    def route(logits=p, dtype=1, select=None, T=4, E=8, K=2, score=0, ids=p, scores=p):
        return L.ep_route(logits, dtype, select, T, E, K, score, 1, 1.0, ids, scores, None)

    assert route(T=0, logits=None, ids=None, scores=None) == _abi.EP_OK
    for kw in (dict(dtype=2), dict(T=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=9), dict(score=2),
               dict(logits=None), dict(ids=None), dict(scores=None), dict(E=128, K=65)):
        assert route(**kw) == bad, kw
    assert route(T=1 << 40) == cap
    for kw in (dict(logits=p + 2), dict(select=p + 1), dict(ids=p + 2), dict(scores=p + 1)):
        assert route(**kw) == al, kw

    def back(grad=p, logits=p, ids=p, out=p, T=4):
        return L.ep_route_backward(grad, logits, 0, ids, T, 8, 2, 1, 0, 1.0, out, None)

    assert back(T=0) == _abi.EP_OK
    for kw in (dict(grad=None), dict(logits=None), dict(ids=None), dict(out=None)):
        assert back(**kw) == bad, kw
    assert back(out=p + 1) == al

    def quant(x=p, rows=4, cols=128, per=4, codes=p, scales=p, ts=None, fmt=0):
        q = _abi.EpFp4(codes, scales, ts, fmt)
        a = L.ep_quantize_fp4(x, rows, cols, per, C.byref(q), None)
        assert a == L.ep_dequantize_fp4(C.byref(q), rows, cols, per, x, 0, None)
        return a

    assert quant(rows=0, x=None, codes=None, scales=None) == _abi.EP_OK
    for kw in (dict(x=None), dict(codes=None), dict(scales=None), dict(cols=64), dict(cols=0),
               dict(rows=-1), dict(per=0), dict(fmt=2), dict(ts=p)):
        assert quant(**kw) == bad, kw
    for kw in (dict(x=p + 8), dict(codes=p + 8), dict(scales=p + 4), dict(ts=p + 2, fmt=1)):
        assert quant(**kw) == al, kw
    assert quant(rows=1 << 31) == cap
    q = _abi.EpFp4(p, p, None, 0)
    assert L.ep_dequantize_fp4(C.byref(q), 4, 128, 4, p, 3, None) == bad
    assert L.ep_quantize_fp4(p, 4, 128, 4, None, None) == bad
    assert L.ep_dispatch_fp4(None, p, p, p, 1, 1, C.byref(q), None, None) == bad
    assert L.ep_expert_gemm_fp4(None, C.byref(q), C.byref(q), 128, 128, p, None) == bad
    assert L.ep_expert_glu_fp4(None, C.byref(q), C.byref(q), 128, 128, 0, p, None, None) == bad
    assert L.ep_expert_glu_fp4(None, C.byref(q), C.byref(q), 128, 128, 9, p, None, None) == bad
    assert L.ep_moe_layer(None, p, p, p, 1, p, p, 128, 0, p, 0, p, 1 << 20, None) == bad
    assert L.ep_moe_layer_fp4(None, p, p, p, 1, C.byref(q), C.byref(q), 128, 0, p, 0, p, 1 << 20,
                              None) == bad
    assert L.ep_moe_layer_workspace_bytes(None, 1, 128) == 0


def test_struct_matches_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no gcc")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "ep.h"', "int main(void) {",
             'printf("%zu\\n", sizeof(ep_fp4));']
    lines += [f'printf("%zu\\n", offsetof(ep_fp4, {f}));' for f, _ in _abi.EpFp4._fields_]
    src, exe = tmp_path / "m.c", tmp_path / "m"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), src, "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [C.sizeof(_abi.EpFp4)] + [getattr(_abi.EpFp4, f).offset for f, _ in _abi.EpFp4._fields_]


def test_the_tests_own_format():
    """The reference quantisation against numbers worked out by hand."""
    x = torch.zeros((1, 128), dtype=torch.float64)
    x[0, :8] = torch.tensor([6.0, 0.25, 0.75, 1.25, 2.5, 5.0, -3.5, -0.1])
    q, s = F4.quantize(x, "mx")
    assert s[0].tolist() == [127, 0, 0, 0]                 # floor(log2 6) - 2 = 0
    assert q[0, :8].tolist() == [7, 0, 2, 2, 4, 6, 14, 0]  # ties to the even code
    q, s = F4.quantize(x, "nv")
    assert s[0, 0] == 0x38 and q[0, :8].tolist() == [7, 0, 2, 2, 4, 6, 14, 0]   # 6 / 6 = 1
    assert F4.values(q, s, "nv")[0, :8].tolist() == [6, 0, 1, 1, 2, 4, -4, 0]
    x[0, 0] = float("nan")
    q, s = F4.quantize(x, "mx")
    assert s[0, 0] == 255 and (q[0, :32] == 0).all()
