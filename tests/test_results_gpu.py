"""Results of a dispatch: fields that are views of the workspace, made when they are asked for."""
import copy
import dataclasses

import pytest
import torch

import combine_topk_ids_expert_gb300 as ep

pytestmark = pytest.mark.gpu


def dispatched(layout="strided"):
    buf = ep.Buffer(32, 256, 8, 2, 2, layout=layout)
    ids = torch.randint(0, 8, (20, 2), device="cuda", dtype=torch.int32)
    x = torch.randn((20, 256), device="cuda").bfloat16()
    return buf, buf.dispatch(x, torch.rand((20, 2), device="cuda"), ids)


@pytest.mark.parametrize("layout", ["strided", "packed"])
def test_fields(layout):
    buf, d = dispatched(layout)
    assert isinstance(d, ep.DispatchResult) and isinstance(d.layout, ep.Layout)
    lead = (2 * 40,) if layout == "packed" else (2, 40)
    assert d.recv_x.shape == (*lead, 256) and d.recv_x.dtype == torch.bfloat16
    assert d.recv_scores.shape == lead and d.recv_src.shape == lead
    assert d.recv_x is d.recv_x
    names = [f.name for f in dataclasses.fields(d.layout)]
    assert names == [f.name for f in dataclasses.fields(ep.Layout)]
    assert all(getattr(d.layout, n) is not None for n in names)
    assert d.layout.pos.shape == (20, 2) and int(d.layout.tokens_per_expert.sum()) == 40
    assert d.layout.num_tokens == 20 and d.layout.rank_stride == 40
    with pytest.raises(AttributeError, match="nothing"):
        d.nothing
    buf.close()


def test_copies_and_replacements():
    buf, d = dispatched()
    assert torch.equal(copy.copy(d).recv_src, d.recv_src)
    y = torch.zeros(1)
    e = dataclasses.replace(d, recv_x=y)
    assert e.recv_x is y and torch.equal(e.recv_scores, d.recv_scores)
    assert "recv_src" in repr(d) and "rank_stride" in repr(d.layout)
    buf.close()


def test_views_outlive_the_buffer():
    buf, d = dispatched()
    torch.cuda.synchronize()
    n = int(d.layout.rows_per_rank.sum())
    buf.close()
    del buf
    assert d.recv_src.numel() == 80 and n == 40
