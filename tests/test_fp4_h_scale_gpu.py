"""What the gated block leaves quantised: against the quantisation, by its definition, of the block in 64
bits, with and without a scale of h's own."""
import pytest
import torch

import fp4_util as F4
import combine_topk_ids_expert_gb300 as ep
from test_fp4_gpu import Case, act64, glu_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,h_scale", [("mx", None), ("nv", None), ("nv", 0.37), ("nv", 2.0 ** -9),
                                         ("nv", 0.0043)])
@pytest.mark.parametrize("kernel", ["1", "2"])
@pytest.mark.parametrize("T,D,F,E,K", [(130, 384, 256, 3, 1), (301, 512, 384, 5, 3)])
def test_h_on_its_own_scale(T, D, F, E, K, kernel, fmt, h_scale, monkeypatch):
    monkeypatch.setenv("EP_GEMM_KERNEL", kernel)
    c = Case(T, D, E, K, fmt, seed=T)
    w, wv = c.weights(E, 2 * F, D, tensor_scale=fmt == "nv")
    ts = None if h_scale is None else torch.tensor([h_scale], device="cuda")
    gh = 1.0 if ts is None else float(ts)
    q = c.buf.expert_glu_fp4(c.d.recv_x, w, quantize=True, h_scale=ts)
    n = F4.BLOCK[fmt]
    scales = ep.untile_fp4_scales(q.scales, q.rows).cpu()
    codes = F4.unpack(q.codes)
    for e, lo, m in c.spans:
        x = c.x[lo:lo + m]
        g, u = x @ wv[e][:F].T, x @ wv[e][F:].T
        want = act64(g, "silu") * u
        bound = glu_bound(x, wv[e][:F], wv[e][F:], g, u, "silu").cpu()
        want = want.cpu()
        sc = scales[lo:lo + m]
        # The block's scale is that of an amax within the bound.
        low = F4.quantize((want.abs() - bound).clamp(min=0), fmt, gh)[1]
        high = F4.quantize(want.abs() + bound, fmt, gh)[1]
        assert ((sc >= low) & (sc <= high)).all()
        # And each code the nearest to a number within the bound, on that scale.
        unit = F4.values(torch.full((m, F), 2), sc, fmt, gh).unflatten(-1, (-1, n))
        got = F4.values(codes[lo:lo + m], sc, fmt, gh).unflatten(-1, (-1, n))
        there = unit > 0
        unit = torch.where(there, unit, 1.0)
        a = want.unflatten(-1, (-1, n)) / unit
        slack = bound.unflatten(-1, (-1, n)) / unit
        near = a.clamp(-6, 6)
        half = torch.where(near.abs() + slack < 2, 0.25, torch.where(near.abs() + slack < 4, 0.5, 1.0))
        assert (((got / unit - near).abs() <= half + slack) | ~there).all()
        assert (got[~there] == 0).all()
        # Values in the large: as far from h as its quantisation is.
        if m * F > 1000 and gh < 0.1:
            ref = F4.values(*F4.quantize(want, fmt, gh), fmt, gh)
            v = got.flatten(-2)
            assert abs(float((v - want).norm() / (ref - want).norm()) - 1) < 0.02
    assert c.buf.device_error() == 0
    c.buf.close()
