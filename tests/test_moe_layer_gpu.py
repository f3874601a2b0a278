"""The layer for a few tokens against a plain one in 64 bits."""
import pytest
import torch

import combine_topk_ids_expert_gb300 as ep
import fp4_util as F4
from test_fp4_gpu import act64, gen, make_ids

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "mx", "nv"]
BF16 = 2.0 ** -8      # half a step of bf16, relative


class Layer:
    def __init__(self, D, F, E, K, fmt, N=64, R=1, seed=0, tensor_scale=True):
        self.D, self.F, self.E, self.K, self.fmt = D, F, E, K, fmt
        self.buf = ep.Buffer(N, D, E, R, K)
        g = gen(seed)
        self.w, self.v = [], []
        for rows, cols in ((2 * F, D), (D, F)):
            if fmt == "bf16":
                w = (torch.randn((E, rows, cols), device="cuda", generator=g) * cols ** -0.5).bfloat16()
                v = w.double()
            else:
                codes, sc = F4.random_fp4(g, (E, rows), cols, fmt, cols ** -0.5)
                ts = None
                if fmt == "nv" and tensor_scale:
                    ts = torch.rand(E, device="cuda", generator=g) + 0.5
                w = ep.FP4(codes, ep.tile_fp4_scales(sc), fmt, ts)
                v = F4.values(F4.unpack(codes.view(-1, cols // 2)), sc.view(-1, sc.shape[-1]), fmt)
                v = v.cuda().view(E, rows, cols)
                if ts is not None:
                    v = v * ts.double()[:, None, None]
            self.w.append(w)
            self.v.append(v)

    def run(self, x, scores, ids, **kw):
        return self.buf.moe_layer(x, scores, ids, *self.w, **kw)

    def rest(self, x, h=False):
        """What the digits (bf16 weights: h's two terms) may leave of x [n, cols], bf16 values, or
        of h."""
        if self.fmt == "bf16":
            return x.abs() * 2.0 ** -16 if h else torch.zeros_like(x)
        n = F4.BLOCK[self.fmt]
        block = x.abs().unflatten(-1, (-1, n)).amax(-1, keepdim=True).expand(-1, -1, n).flatten(-2)
        rest = block * 2.0 ** -14 if h else \
            torch.where(x.abs() * 16 >= block, 0.0, block * 2.0 ** -11)
        if self.fmt == "nv":
            rest = torch.maximum(rest, x.abs().amax(-1, keepdim=True) * 2.0 ** -28)
        return rest

    def sums(self, x, w, h=False):
        """n 2^-23 sum |x w| for any order, an eighth more for the lower digits' own sums, and
        the digits' rest."""
        return (1.2 * x.shape[-1] * 2.0 ** -23) * (x.abs() @ w.abs().T) + self.rest(x, h) @ w.abs().T

    def reference(self, x, scores, ids, act):
        """(result, how far it may be off before its last rounding) in 64 bits."""
        F = self.F
        out = torch.zeros((x.shape[0], self.D), dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(out)
        for e in range(self.E):
            t, k = (ids == e).nonzero(as_tuple=True)
            if not len(t):
                continue
            xe, wg, wu, wd = x[t].double(), self.v[0][e][:F], self.v[0][e][F:], self.v[1][e]
            g, u = xe @ wg.T, xe @ wu.T
            h = act64(g, act) * u
            dg, du = self.sums(xe, wg), self.sums(xe, wu)
            # |act'| <= 1.13, |act(g)| <= |g|; the activation's own arithmetic 2^-18.
            dh = 1.13 * dg * u.abs() + g.abs() * du + 1.13 * dg * du + 2.0 ** -18 * h.abs()
            y = h @ wd.T
            dy = dh @ wd.abs().T + self.sums(h.abs() + dh, wd, h=True)
            s = scores[t, k].double()[:, None]
            out.index_add_(0, t, s * y)
            bound.index_add_(0, t, s.abs() * (dy + 2.0 ** -20 * y.abs()))
        return out, bound

    def check(self, T, act="silu", out_dtype=torch.bfloat16, seed=1, drop=0.1, ids=None, scale=1.0):
        g = gen(seed)
        x = (torch.randn((T, self.D), device="cuda", generator=g) * scale).bfloat16()
        scores = torch.rand((T, self.K), device="cuda", generator=g)
        ids = make_ids(T, self.E, self.K, seed, drop) if ids is None else ids
        got = self.run(x, scores, ids, act=act, out_dtype=out_dtype)
        want, bound = self.reference(x, scores, ids, act)
        err = (got.double() - want).abs()
        last = BF16 if out_dtype == torch.bfloat16 else 2.0 ** -24
        assert (err <= bound + last * (want.abs() + bound)).all()
        # The last rounding is at most 2^-8 relative in each element; what the digits leave, at most
        # 2^-11 of a block's largest in the elements below a sixteenth of it, goes both ways and is
        # a small part of 2^-11 in the root mean square.
        if want.norm() > 0:
            assert err.norm() <= (last + 2.0 ** -11) * want.norm()
        assert torch.equal(got, self.run(x, scores, ids, act=act, out_dtype=out_dtype))
        assert self.buf.device_error() == 0
        return got


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,D,F,E,K", [
    (1, 128, 128, 1, 1),
    (1, 512, 256, 8, 2),
    (2, 384, 128, 5, 3),
    (13, 640, 384, 8, 2),
    (16, 256, 128, 1, 1),
    (17, 256, 128, 1, 1),
    (64, 256, 256, 2, 1),
    (64, 384, 128, 16, 8),
    (7, 256, 128, 300, 64),
    (3, 1024, 2048, 1024, 4),
])
def test_layer(fmt, T, D, F, E, K):
    if E * D * F > 2 ** 29 and fmt != "nv":
        E = 64
    layer = Layer(D, F, E, K, fmt, seed=T)
    layer.check(T, act="gelu" if T % 2 else "silu",
                out_dtype=torch.float32 if D == 256 else torch.bfloat16)
    layer.buf.close()


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_sizes(fmt):
    """One token and 16 on the shapes of a decode batch: several units to a CTA."""
    layer = Layer(2048, 1024, 32, 8, fmt, seed=3)
    for T in (1, 16, 64):
        layer.check(T, seed=T, drop=0.0)
    layer.buf.close()


@pytest.mark.parametrize("sms", [1, 2, 3, 5, 8, 150])
@pytest.mark.parametrize("fmt", FORMATS)
def test_grids(fmt, sms, monkeypatch):
    """SM budgets that give one CTA all units, or clusters of different sizes."""
    monkeypatch.setenv("EP_NUM_SMS", str(sms))
    layer = Layer(1024, 256, 4, 2, fmt, seed=sms)
    layer.check(5, seed=sms)
    layer.buf.close()


@pytest.mark.parametrize("fmt", FORMATS)
def test_no_experts_and_bad_ids(fmt):
    layer = Layer(256, 128, 4, 2, fmt)
    none = torch.full((9, 2), -1, dtype=torch.int32, device="cuda")
    x = torch.randn((9, 256), device="cuda").bfloat16()
    scores = torch.rand((9, 2), device="cuda")
    out = torch.full((9, 256), 3.0, device="cuda")
    assert (layer.run(x, scores, none, out=out) == 0).all()
    assert layer.buf.device_error() == 0
    some = none.clone()
    some[4] = torch.tensor([2, 77], dtype=torch.int32)
    some[5] = torch.tensor([-9, 0], dtype=torch.int32)
    out = layer.run(x, scores, some, out_dtype=torch.float32)
    assert layer.buf.device_error() == ep.EP_DEVERR_BAD_ID
    clean = torch.where((some < 0) | (some >= 4), -1, some)
    assert torch.equal(out, layer.run(x, scores, clean, out_dtype=torch.float32))
    assert (out[[0, 1, 2, 3, 6, 7, 8]] == 0).all() and (out[4:6].abs().sum(1) > 0).all()
    empty = layer.run(x[:0], scores[:0], none[:0])
    assert empty.shape == (0, 256)
    layer.buf.close()


@pytest.mark.parametrize("fmt", FORMATS)
def test_same_expert_twice(fmt):
    layer = Layer(256, 128, 4, 4, fmt)
    ids = torch.tensor([[1, 1, 1, 2], [0, 0, -1, 0]], dtype=torch.int32, device="cuda")
    layer.check(2, ids=ids)
    layer.buf.close()


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_rows_stay_their_own(fmt):
    layer = Layer(512, 256, 2, 1, fmt)
    T = 24
    x = torch.randn((T, 512), device="cuda", generator=gen(1)).bfloat16()
    ids = (torch.arange(T, device="cuda") % 2).to(torch.int32)[:, None].contiguous()
    scores = torch.ones((T, 1), device="cuda")
    clean = layer.run(x, scores, ids)
    x[3, 77], x[8, 500], x[20, 0] = float("nan"), float("inf"), float("-inf")
    out = layer.run(x, scores, ids)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[3, 8, 20]] = True
    assert not torch.isfinite(out[bad]).any()
    assert torch.equal(out[~bad], clean[~bad])
    layer.buf.close()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("scale", [2.0 ** -100, 1e-6, 300.0, 2.0 ** 50])
def test_scales_of_rows(fmt, scale):
    """Rows far from 1: the digits' powers of two follow them. (The down projection sees h.)"""
    layer = Layer(384, 128, 2, 1, fmt, tensor_scale=False)
    T = 5
    x = torch.randn((T, 384), device="cuda", generator=gen(5)).bfloat16()
    x *= scale
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    got = layer.run(x, torch.ones((T, 1), device="cuda"), ids, out_dtype=torch.float32)
    want, bound = layer.reference(x, torch.ones((T, 1), device="cuda"), ids, "silu")
    # 2^-120: h and its products may be subnormal, or nothing.
    assert ((got.double() - want).abs() <= bound + 2.0 ** -24 * want.abs() + 2.0 ** -120).all()
    layer.buf.close()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_uneven_blocks(fmt):
    """Blocks from 2^-24 to 2^20 in a row; weights of the large ones zero, so that the small ones
    are the result."""
    D, F = 512, 128
    layer = Layer(D, F, 1, 1, fmt, tensor_scale=False)
    n = F4.BLOCK[fmt]
    x = torch.randn((4, D), device="cuda", generator=gen(6))
    exps = torch.randint(-24, 21, (4, D // n), device="cuda", generator=gen(7)).float()
    x = (x.view(4, -1, n) * torch.exp2(exps)[..., None]).view(4, D).bfloat16()
    scores, ids = torch.ones((4, 1), device="cuda"), torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    got = layer.run(x, scores, ids, out_dtype=torch.float32)
    want, bound = layer.reference(x, scores, ids, "silu")
    assert ((got.double() - want).abs() <= bound + 2.0 ** -24 * want.abs()).all()
    layer.buf.close()


def test_agrees_with_the_three_calls():
    """bf16: dispatch, block, combine on the same inputs agree within their roundings."""
    layer = Layer(512, 256, 8, 2, "bf16", seed=4)
    T = 33
    x = torch.randn((T, 512), device="cuda", generator=gen(8)).bfloat16()
    scores, ids = torch.rand((T, 2), device="cuda"), make_ids(T, 8, 2, 9)
    d = layer.buf.dispatch(x, scores, ids)
    three = layer.buf.combine(layer.buf.expert_ffn(d.recv_x, *layer.w), scores)
    pos = d.layout.pos.clone()
    one = layer.run(x, scores, ids)
    assert torch.equal(d.layout.pos, pos)          # the layout is left alone
    want, bound = layer.reference(x, scores, ids, "silu")
    y_rounding = BF16 * 3 * want.abs().amax()      # the pairs' results in bf16
    assert ((three.double() - one.double()).abs() <= 2 * bound + 2 * BF16 * want.abs() + y_rounding).all()
    layer.buf.close()


@pytest.mark.parametrize("fmt", FORMATS)
def test_back_to_back_and_captured(fmt):
    """Calls that follow one another without a wait, on new tokens and experts each, and replays
    of a captured pair of layers."""
    a, b = Layer(512, 256, 8, 2, fmt, seed=1), Layer(512, 128, 8, 2, fmt, seed=2)
    T = 6
    g = gen(3)
    xs = [torch.randn((T, 512), device="cuda", generator=g).bfloat16() for _ in range(6)]
    ids = [make_ids(T, 8, 2, 20 + i) for i in range(6)]
    scores = torch.rand((T, 2), device="cuda", generator=g)

    def two(x, i):
        return b.run(a.run(x, scores, i), scores, i)

    alone = []
    for x, i in zip(xs, ids):
        alone.append(two(x, i))
        torch.cuda.synchronize()
    chained = [two(x, i) for x, i in zip(xs, ids)]
    assert all(torch.equal(p, q) for p, q in zip(alone, chained))
    x, i = xs[0].clone(), ids[0].clone()
    two(x, i)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = two(x, i)
    for n in (3, 1, 5):
        x.copy_(xs[n])
        i.copy_(ids[n])
        graph.replay()
        assert torch.equal(out, alone[n])
    del graph
    assert a.buf.device_error() == 0 and b.buf.device_error() == 0
    a.buf.close()
    b.buf.close()


def test_streams():
    """Two layers at once on two streams, results on a stream of the caller's choice."""
    a, b = Layer(1024, 512, 16, 4, "mx", seed=1), Layer(1024, 512, 16, 4, "bf16", seed=2)
    T = 8
    x = torch.randn((T, 1024), device="cuda", generator=gen(1)).bfloat16()
    ids, scores = make_ids(T, 16, 4, 2), torch.rand((T, 4), device="cuda")
    want = a.run(x, scores, ids), b.run(x, scores, ids)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        got = a.run(x, scores, ids, stream=s), b.run(x, scores, ids, stream=t)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a.buf.close()
    b.buf.close()


def test_refusals():
    layer = Layer(256, 128, 4, 2, "nv")
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    scores = torch.zeros((4, 2), device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    run = layer.buf.moe_layer
    w1, w2 = layer.w
    with pytest.raises(ValueError, match="weights"):
        run(x, scores, ids, w2, w1)
    with pytest.raises(TypeError, match="both"):
        run(x, scores, ids, w1, layer.v[1].bfloat16())
    with pytest.raises(ValueError, match="x, scores and ids"):
        run(x[:, :128].contiguous(), scores, ids, w1, w2)
    with pytest.raises(ValueError, match="act"):
        run(x, scores, ids, w1, w2, act="relu")
    with pytest.raises(TypeError):
        run(x.float(), scores, ids, w1, w2)
    with pytest.raises(ValueError, match="out"):
        run(x, scores, ids, w1, w2, out=x[:2])
    many = torch.zeros((65, 256), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ep.EpError) as e:
        run(many, torch.zeros((65, 2), device="cuda"),
            torch.zeros((65, 2), dtype=torch.int32, device="cuda"), w1, w2)
    assert e.value.status == ep._abi.EP_ERR_CAPACITY
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ep.EpError) as e:
        ep.ep_moe_layer_fp4(layer.buf.handle, x, scores, ids, 4, w1, w2, 128, 0, x.clone(), small)
    assert e.value.status == ep._abi.EP_ERR_WORKSPACE
    layer.buf.close()
