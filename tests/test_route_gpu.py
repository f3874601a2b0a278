"""The router on the GPU against its definition in 64 bits, and its gradient against the formula's
and against differences."""
import math

import pytest
import torch

import combine_topk_ids_expert_gb300 as ep

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def choose(select, K):
    """Chosen one after the other: the lowest index of the largest value left."""
    left = select.double().clone()
    left[torch.isnan(left)] = -math.inf
    out = []
    col = torch.arange(left.shape[1], device=left.device)
    for _ in range(K):
        most = left.amax(1, keepdim=True)
        first = torch.where(left == most, col, left.shape[1]).amin(1)
        first = torch.where(most[:, 0] == -math.inf, -1, first)
        out.append(first)
        left[col == first[:, None]] = -math.inf
    return torch.stack(out, 1)


def scores_of(logits, ids, score, normalize, scale):
    """The scores in 64 bits (autograd follows)."""
    v = logits
    p = torch.special.expit(v) if score == "sigmoid" else torch.softmax(v, 1)
    here = ids >= 0
    c = torch.where(here, p.gather(1, ids.clamp(min=0)), 0.0)
    if normalize:
        total = c.sum(1, keepdim=True)
        c = torch.where(total > 0, c / torch.where(total > 0, total, 1.0), 0.0)
    return scale * c


KINDS = [(s, n) for s in ("softmax", "sigmoid") for n in (True, False)]


@pytest.mark.parametrize("score,normalize", KINDS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 5, 5), (70, 33, 4), (257, 64, 8), (64, 256, 8),
                                   (9, 1000, 64), (5, 1024, 1), (40, 160, 40)])
def test_route(T, E, K, dtype, score, normalize):
    logits = (torch.randn((T, E), device="cuda", generator=gen(T + E)) * 2).to(dtype)
    ids, scores = ep.route(logits, K, score, normalize, scale=2.5)
    want = choose(logits, K)
    assert torch.equal(ids.long(), want)
    ref = scores_of(logits.double(), want, score, normalize, 2.5)
    # exp 2 ulp, its argument's rounding at most |l - m| 2^-24, a sum of E (n 2^-24 relative),
    # a division and two products: all within 2^-23 (8 + |l - m| + E).
    spread = (logits.float().amax(1) - logits.float().amin(1)).clamp(min=0)[:, None].double()
    assert ((scores.double() - ref).abs() <= ref * (8 + spread + E) * 2.0 ** -23).all()


def test_ties_and_masks():
    T, E, K = 6, 40, 4
    logits = torch.zeros((T, E), device="cuda")
    logits[1, ::2] = -0.0
    select = logits.clone()
    select[2, :37] = -math.inf          # three left
    select[3] = -math.inf               # nothing left
    select[4] = torch.finfo(torch.float32).min
    select[5, 3] = math.nan
    ids, scores = ep.route(logits, K, select=select)
    assert ids.tolist() == [[0, 1, 2, 3], [0, 1, 2, 3], [37, 38, 39, -1], [-1] * 4, [0, 1, 2, 3],
                            [0, 1, 2, 4]]
    assert torch.allclose(scores[:2], torch.full((2, 4), 0.25, device="cuda"))
    third = torch.tensor([1 / 3] * 3 + [0.0], device="cuda")
    assert torch.allclose(scores[2], third) and scores[3].tolist() == [0.0] * 4
    for kind in KINDS:
        ids, scores = ep.route(torch.full((2, E), -math.inf, device="cuda"), K, *kind)
        assert (ids == -1).all() and (scores == 0).all()
        ids, scores = ep.route(torch.full((2, E), -math.inf, device="cuda"), K, *kind,
                               select=torch.zeros((2, E), device="cuda"))
        assert ids[0].tolist() == [0, 1, 2, 3] and (scores == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_logits(score):
    """Normalised scores of logits whose probabilities underflow fp32."""
    logits = torch.tensor([[0.0] * 4 + [-200.0, -201.0, -90.0, -1000.0]], device="cuda")
    select = torch.tensor([[-math.inf] * 4 + [4.0, 3.0, 2.0, 1.0]], device="cuda")
    _, scores = ep.route(logits, 2, score, select=select)
    want = torch.softmax(torch.tensor([-200.0, -201.0], dtype=torch.float64), 0)
    assert torch.allclose(scores[0].cpu().double(), want, rtol=1e-6)
    _, scores = ep.route(torch.tensor([[300.0, 80.0, -5.0]], device="cuda"), 3, "sigmoid")
    want = torch.special.expit(torch.tensor([300.0, 80.0, -5.0], dtype=torch.float64))
    assert torch.allclose(scores[0].cpu().double(), want / want.sum(), rtol=1e-6)


@pytest.mark.parametrize("score,normalize", KINDS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (33, 20, 3), (130, 64, 8), (64, 256, 8), (7, 1000, 64),
                                   (12, 300, 40)])
def test_backward(T, E, K, dtype, score, normalize):
    g = gen(T)
    logits = (torch.randn((T, E), device="cuda", generator=g) * 2).to(dtype)
    select = logits.float().masked_fill(torch.rand((T, E), device="cuda", generator=g) < 0.2,
                                        -math.inf)
    if T > 1:
        select[0] = -math.inf
    ids, _ = ep.route(logits, K, score, normalize, select=select, scale=1.5)
    grad = torch.randn((T, K), device="cuda", generator=g)
    got = ep.route_backward(grad, logits, ids, score, normalize, scale=1.5)
    assert got.dtype == dtype
    leaf = logits.double().requires_grad_(True)
    (scores_of(leaf, ids.long(), score, normalize, 1.5) * grad.double()).sum().backward()
    want = leaf.grad
    # c - sum c s cancels: the error counts against the largest |c| of the row (times the weight),
    # (K + E) roundings of the sums, exp's and the factors'. bf16: half a step more.
    p = torch.special.expit(leaf) if score == "sigmoid" else torch.softmax(leaf, 1)
    if normalize:
        here = (ids >= 0).double()
        chosen = torch.zeros_like(p).scatter_add_(1, ids.long().clamp(min=0), here).clamp(max=1)
        total = (p * chosen).sum(1, keepdim=True)
        p = p * chosen / torch.where(total > 0, total, 1.0)
    most = 1.5 * grad.abs().amax(1, keepdim=True).double()
    # 2^-48: what the 64-bit reference leaves of terms that cancel where nothing is chosen.
    bound = p.detach() * most * (K + E + 40) * 2.0 ** -22 + most * 2.0 ** -48
    if dtype == torch.bfloat16:
        bound = bound + want.abs() * 2.0 ** -8
    assert ((got.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("score,normalize", KINDS)
def test_backward_against_differences(score, normalize):
    """(s(l + d) - s(l - d)) / 2d in 64 bits through the plain scores, at d = 2^-10: off by
    d^2 / 6 times a third derivative of at most 8 (a product of probabilities below 1)."""
    T, E, K = 4, 12, 3
    g = gen(3)
    logits = torch.randn((T, E), device="cuda", generator=g)
    ids, _ = ep.route(logits, K, score, normalize)
    grad = torch.randn((T, K), device="cuda", generator=g)
    got = ep.route_backward(grad, logits, ids, score, normalize).double()
    d = 2.0 ** -10
    for e in range(E):
        up, down = logits.double().clone(), logits.double().clone()
        up[:, e] += d
        down[:, e] -= d
        s = [scores_of(v, ids.long(), score, normalize, 1.0) * grad.double() for v in (up, down)]
        want = (s[0] - s[1]).sum(1) / (2 * d)
        assert ((got[:, e] - want).abs() <= grad.abs().sum(1) * (8 * d * d / 6 + 2.0 ** -18)).all()


@pytest.mark.parametrize("score,normalize", KINDS)
def test_backward_same_id_twice_and_empty_slots(score, normalize):
    logits = torch.randn((2, 6), device="cuda", generator=gen(8))
    ids = torch.tensor([[2, 2, -1, 2], [7, -1, -5, 0]], dtype=torch.int32, device="cuda")
    grad = torch.randn((2, 4), device="cuda", generator=gen(9))
    got = ep.route_backward(grad, logits, ids, score, normalize)
    leaf = logits.double().requires_grad_(True)
    clean = torch.where((ids >= 0) & (ids < 6), ids, -1).long()
    (scores_of(leaf, clean, score, normalize, 1.0) * grad.double()).sum().backward()
    assert torch.allclose(got.double(), leaf.grad, atol=1e-6)
    again = ep.route_backward(grad, logits, ids, score, normalize)
    assert torch.equal(got, again)


def test_empty_and_streams():
    ids, scores = ep.route(torch.empty((0, 8), device="cuda"), 2)
    assert ids.shape == scores.shape == (0, 2)
    assert ep.route_backward(scores, torch.empty((0, 8), device="cuda"), ids).shape == (0, 8)
    s = torch.cuda.Stream()
    logits = torch.randn((4096, 64), device="cuda", generator=gen(1))
    here = ep.route(logits, 4)
    s.wait_stream(torch.cuda.current_stream())
    there = ep.route(logits, 4, stream=s)
    s.synchronize()
    assert torch.equal(here[0], there[0]) and torch.equal(here[1], there[1])


def test_routed_layer_dispatches():
    """Router, dispatch, combine and back: padded tokens route nowhere and get zero rows."""
    T, D, E, K = 20, 64, 8, 2
    buf = ep.Buffer(T, D, E, 2, K, dtype=torch.float32)
    logits = torch.randn((T, E), device="cuda", generator=gen(2))
    select = logits.clone()
    select[15:] = -math.inf
    ids, scores = ep.route(logits, K, select=select)
    x = torch.randn((T, D), device="cuda", generator=gen(3))
    d = buf.dispatch(x, scores, ids)
    y = d.recv_x.clone()
    out = buf.combine(y, scores)
    assert torch.allclose(out[:15], x[:15], atol=1e-6) and (out[15:] == 0).all()
    _, gs = buf.combine_backward(torch.randn((T, D), device="cuda"), y, scores)
    gl = ep.route_backward(gs, logits, ids)
    assert (gl[15:] == 0).all() and gl[:15].abs().sum() > 0
    assert buf.device_error() == 0
    buf.close()


@pytest.mark.parametrize("T,E,K", [(40, 8, 4), (40, 30, 30), (60, 100, 12), (60, 256, 8),
                                   (60, 256, 64), (30, 400, 40), (30, 512, 10), (20, 900, 33)])
@pytest.mark.parametrize("levels", [1, 2, 5])
def test_many_equal_values(T, E, K, levels):
    """Runs of equal values in a lane, over lanes and over the 32nd slot; both zeros, infinities."""
    g = gen(E + K + levels)
    select = torch.randint(0, levels, (T, E), device="cuda", generator=g).float()
    select[::3] *= -0.0
    select[1, E // 3:E // 3 + 4] = math.inf
    select[2, E // 2:] = -math.inf
    select[4, ::2] = math.nan
    logits = torch.randn((T, E), device="cuda", generator=g)
    ids, scores = ep.route(logits, K, "sigmoid", select=select)
    want = choose(select, K)
    assert torch.equal(ids.long(), want)
    by_logits, _ = ep.route(select.bfloat16(), K, "sigmoid")
    assert torch.equal(by_logits.long(), choose(select.bfloat16(), K))
    assert torch.isfinite(scores).all()
