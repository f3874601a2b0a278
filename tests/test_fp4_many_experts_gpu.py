"""The experts' products in 4 bits over many experts of a few rows each: tiles of single SMs and of pairs
against 64 bits, and the same bits from both and from the rule between them."""
import pytest
import torch

from test_fp4_gpu import BF16, Case, act64, glu_bound, make_ids, product_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T,D,F,E,K", [(16, 512, 256, 256, 8), (70, 256, 256, 256, 8), (500, 256, 128, 64, 4),
                                       (3000, 256, 256, 64, 4), (40, 128, 256, 1024, 2)])
def test_many_experts(T, D, F, E, K, fmt, monkeypatch):
    results = {}
    for kernel in ("1", "2", "0"):
        monkeypatch.setenv("EP_GEMM_KERNEL", kernel)
        # Some experts have most of the rows, and some none.
        ids = make_ids(T, E, K, T, drop=0.1)
        ids[:, 0] = torch.arange(T, device="cuda", dtype=torch.int32) % 3
        ids[:, 1:][ids[:, 1:] < 3] = -1
        c = Case(T, D, E, K, fmt, seed=T, ids=ids)
        w, wv = c.weights(E, F, D, tensor_scale=fmt == "nv")
        w1, w1v = c.weights(E, 2 * F, D, tensor_scale=fmt == "nv")
        n = max(lo + m for _, lo, m in c.spans)
        y = c.buf.expert_gemm_fp4(c.d.recv_x, w)[:n]
        h = c.buf.expert_glu_fp4(c.d.recv_x, w1)[:n]
        q = c.buf.expert_glu_fp4(c.d.recv_x, w1, quantize=True).codes[:n]
        results[kernel] = y, h, q
        assert c.buf.device_error() == 0
        if kernel == "1":
            for e, lo, m in c.spans:
                x = c.x[lo:lo + m]
                want = x @ wv[e].T
                bound = product_bound(x, wv[e]) + (BF16 + 2.0 ** -23) * want.abs()
                assert ((y[lo:lo + m].double() - want).abs() <= bound).all(), (e, m)
                wg, wu = w1v[e][:F], w1v[e][F:]
                g, u = x @ wg.T, x @ wu.T
                want = act64(g, "silu") * u
                bound = glu_bound(x, wg, wu, g, u, "silu") + BF16 * want.abs()
                assert ((h[lo:lo + m].double() - want).abs() <= bound).all(), (e, m)
        c.buf.close()
    for kernel in ("2", "0"):
        assert all(torch.equal(a, b) for a, b in zip(results["1"], results[kernel]))
