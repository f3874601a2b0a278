"""The weight gradients at sizes of several tiles in both directions, on an SM pair (both
sizes multiples of 256) and on one SM, against plain 64-bit products. Bounds as in
test_expert_ffn_gpu.py."""
import pytest
import torch

from test_expert_ffn_gpu import Case, sum_tol

pytestmark = pytest.mark.gpu

F64 = torch.float64

# (T, E, K, din, dout): rows per expert from none to several slices of 64, ragged and whole.
SIZES = [(700, 5, 2, 512, 768), (700, 5, 2, 1024, 512), (64, 2, 1, 768, 768), (333, 9, 2, 256, 1024),
         (450, 3, 2, 512, 384), (450, 3, 1, 384, 512), (200, 4, 2, 192, 256)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_weight_gradients_of_several_tiles(size, dtype, accumulate):
    T, E, K, din, dout = size
    c = Case(93, T, E, K, 1, "zipf", drop=0.1)
    gy, x = c.recv(dout), c.recv(din)
    before = c.randn(E, dout, din).to(dtype)
    got = before.clone()
    c.buf.expert_gemm_backward(gy, x, None, want_x=False, grad_weights=got, accumulate=accumulate)
    ref = before.to(F64) if accumulate else torch.zeros((E, dout, din), dtype=F64, device="cuda")
    tol = torch.zeros_like(ref)
    for e, lo, hi in c.spans:
        a, b = gy[lo:hi].to(F64).T, x[lo:hi].to(F64)
        ref[e] += a @ b
        tol[e] = sum_tol(hi - lo, a.abs() @ b.abs())
    if accumulate:
        tol += 2.0 ** -23 * (ref.abs() + before.to(F64).abs())
    if dtype == torch.bfloat16:
        tol += 2.0 ** -8 * ref.abs()
    bad = (got.to(F64) - ref).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())
    c.done()
