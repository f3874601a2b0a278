"""Each form of the quantising dispatch writes all that it says: its outputs hold other values before,
and a plain dispatch's results come from another buffer."""
import pytest
import torch

import combine_topk_ids_expert_gb300 as ep
import fp4_util as F4
from test_fp4_gpu import gen, make_ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,scaled", [("mx", False), ("nv", False), ("nv", True)])
@pytest.mark.parametrize("layout,R", [("strided", 2), ("packed", 2)])
@pytest.mark.parametrize("form", ["small", "barrier", "kernels"])
@pytest.mark.parametrize("T,N", [(13, 16), (301, 301), (650, 652)])
def test_everything_is_written(form, T, N, layout, R, fmt, scaled, monkeypatch):
    """In one kernel, without a grid barrier and with one, and kernel after kernel."""
    monkeypatch.setenv("EP_DISPATCH_ONEPASS", "0" if form == "kernels" else "1")
    monkeypatch.setenv("EP_DISPATCH_SMALL_PAIRS", "4096" if form == "small" else "0")
    D, E, K = 640, 8, 3
    ids = make_ids(T, E, K, T)
    x = torch.randn((T, D), device="cuda", generator=gen(2)).bfloat16()
    scores = torch.rand((T, K), device="cuda", generator=gen(3))
    ts = torch.tensor([0.0019], device="cuda") if scaled else None
    other = ep.Buffer(N, D, E, R, K, layout=layout)
    plain = other.dispatch(x, scores, ids, N)
    buf = ep.Buffer(N, D, E, R, K, layout=layout)
    # Values that no result has, wherever results go (the barrier's words, which start as zeros, are
    # the library's: only the results' places are filled, by way of a first call's views).
    first = buf.dispatch(x[:1], scores[:1], ids[:1].contiguous(), N)
    lay = first.layout
    first.recv_scores.fill_(float("nan"))
    first.recv_src.fill_(-7)
    pos_all = lay.pos.as_strided((T, K), (K, 1))       # of the call that follows
    pos_all.fill_(-7)
    for t in (lay.tokens_per_expert, lay.expert_offset, lay.rows_per_rank, lay.rank_prefix,
              lay.tokens_in_rank):
        t.fill_(-7)
    d = buf.dispatch_fp4(x, scores, ids, N, format=fmt, tensor_scale=ts)
    for name in ("tokens_per_expert", "expert_offset", "rows_per_rank", "rank_prefix", "tokens_in_rank"):
        assert torch.equal(getattr(d.layout, name), getattr(plain.layout, name)), name
    here = ids.flatten() >= 0
    pos = d.layout.pos.flatten()
    assert torch.equal(pos[here], plain.layout.pos.flatten()[here]) and (pos[~here] < 0).all()
    assert (pos[~here] == plain.layout.pos.flatten()[~here]).all()
    pos = pos[here].long()
    src = torch.arange(T * K, device="cuda")[here]
    assert torch.equal(d.recv_scores.flatten()[pos], scores.flatten()[src])
    assert torch.equal(d.recv_src.flatten()[pos].long(), src)
    codes, scale = F4.quantize(x, fmt, float(ts) if scaled else 1.0)
    token = (src // K).cpu()
    assert torch.equal(F4.unpack(d.recv_x.codes[pos]), codes[token])
    assert torch.equal(ep.untile_fp4_scales(d.recv_x.scales, d.recv_x.rows)[pos].cpu(), scale[token])
    assert buf.device_error() == 0
    for b in (buf, other):
        b.close()
