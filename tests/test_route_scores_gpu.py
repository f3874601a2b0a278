"""The router's scores where the experts are chosen by something else than the logits: a mask, a bias,
numbers of their own; for each type of logits."""
import math

import pytest
import torch

import combine_topk_ids_expert_gb300 as ep
from test_route_gpu import KINDS, choose, gen, scores_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score,normalize", KINDS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["masked", "biased", "unrelated"])
@pytest.mark.parametrize("T,E,K", [(3, 5, 5), (70, 33, 4), (257, 64, 8), (64, 256, 8), (9, 1000, 64),
                                   (40, 160, 40)])
def test_scores_of_selected_experts(T, E, K, kind, dtype, score, normalize):
    g = gen(T + E)
    logits = (torch.randn((T, E), device="cuda", generator=g) * 2).to(dtype)
    select = logits.float()
    if kind == "masked":
        select = select.masked_fill(torch.rand((T, E), device="cuda", generator=g) < 0.4, -math.inf)
        select[T - 1] = -math.inf
    elif kind == "biased":
        select = torch.sigmoid(select) + torch.randn(E, device="cuda", generator=g)
    else:
        select = torch.randn((T, E), device="cuda", generator=g)
    ids, scores = ep.route(logits, K, score, normalize, select=select, scale=1.75)
    want = choose(select, K)
    assert torch.equal(ids.long(), want)
    ref = scores_of(logits.double(), want, score, normalize, 1.75)
    # As for logits that choose by themselves: exp 2 ulp, its argument's rounding at most
    # |l - m| 2^-24, a sum of E, a division and two products: 2^-23 (8 + |l - m| + E).
    spread = (logits.float().amax(1) - logits.float().amin(1))[:, None].double()
    assert ((scores.double() - ref).abs() <= ref * (8 + spread + E) * 2.0 ** -23).all()
    assert (scores[ids < 0] == 0).all()
