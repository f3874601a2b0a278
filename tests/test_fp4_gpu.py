"""Microscaled 4-bit floating point on the GPU: quantisation bit for bit, the quantising dispatch,
and the experts' products against plain ones in 64 bits."""
import pytest
import torch

import combine_topk_ids_expert_gb300 as ep
import fp4_util as F4

pytestmark = pytest.mark.gpu

FORMATS = ["mx", "nv"]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def assert_quantized(q: ep.FP4, x: torch.Tensor, g=1.0):
    """q holds x [rows, cols] exactly as the definition says."""
    codes, scale = F4.quantize(x, q.format, g)
    got = ep.untile_fp4_scales(q.scales, x.shape[0]).cpu()
    assert torch.equal(got, scale)
    assert torch.equal(F4.unpack(q.codes.reshape(x.shape[0], -1)), codes)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols", [(1, 128), (5, 256), (127, 384), (128, 128), (129, 1024),
                                       (333, 640), (1000, 7168)])
def test_quantize(fmt, rows, cols):
    x = torch.randn((rows, cols), device="cuda", generator=gen(rows)).mul_(3).bfloat16()
    x[:, ::61] *= 40
    x[rows // 2] = 0
    q = ep.quantize_fp4(x, fmt)
    assert_quantized(q, x)
    codes, scale = F4.quantize(x, fmt)
    want = F4.values(codes, scale, fmt)
    assert torch.equal(q.dequantize(torch.float32).cpu().double(), want)
    assert torch.equal(q.dequantize().cpu(), want.bfloat16())   # 4 + 4 bits: exact in bf16


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_every_border(fmt):
    """Every bf16 magnitude next to each amax of a few binades: all borders between codes."""
    mantissas = torch.arange(128, 256, dtype=torch.float64)
    values = torch.cat([mantissas * 2.0 ** e for e in range(-14, -6)])     # 2^-7 .. 2
    most = torch.arange(128, 256, dtype=torch.float64) * 2.0 ** -7
    blocks = []
    for m in most:
        v = values[values <= m]
        n = F4.BLOCK[fmt] - 1
        v = torch.nn.functional.pad(v, (0, -len(v) % n)).view(-1, n)
        blocks.append(torch.cat((m.expand(len(v), 1), v), dim=1))
    x = torch.cat(blocks).flatten()
    x = torch.nn.functional.pad(x, (0, -len(x) % 1024)).view(-1, 1024)
    x[:, 1::2] *= -1
    x = x.bfloat16().cuda()
    assert_quantized(ep.quantize_fp4(x, fmt), x)


@pytest.mark.parametrize("g", [1.0, 2.0 ** -9, 0.0123, 3.7, 1e-10])
def test_quantize_tensor_scale(g):
    E, rows, cols = 3, 40, 256
    x = torch.randn((E, rows, cols), device="cuda", generator=gen(1)).bfloat16()
    x[1] *= 100
    ts = torch.tensor([g, 2 * g, g / 3], device="cuda") * 0.01
    q = ep.quantize_fp4(x, "nv", ts)
    scales = ep.untile_fp4_scales(q.scales, E * rows).view(E, rows, -1)
    for e in range(E):
        codes, scale = F4.quantize(x[e], "nv", float(ts[e].double()))
        assert torch.equal(scales[e].cpu(), scale)
        assert torch.equal(F4.unpack(q.codes[e]), codes)
        want = F4.values(codes, scale, "nv", 1.0)
        # The product with g is rounded to fp32, and again to bf16.
        got = q.dequantize(torch.float32)[e].cpu()
        assert torch.equal(got, (want.float() * ts[e].cpu()))
        assert torch.equal(q.dequantize()[e].cpu(), (want.float() * ts[e].cpu()).bfloat16())


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_extremes(fmt):
    """Infinities, NaNs, the largest and the smallest numbers, each in a block of its own."""
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    n = F4.BLOCK[fmt]
    specials = [float("inf"), float("-inf"), float("nan"), 3.3895e38, 2.0 ** -126, 2.0 ** -133,
                -1.0, 1.1755e-38]
    for i, v in enumerate(specials):
        row, block = divmod(i, 256 // n)
        x[row, block * n + 3 * i % n] = v
        x[row, block * n + (3 * i + 1) % n] = 0.5 if i < 3 else 0.0
    q = ep.quantize_fp4(x, fmt)
    assert_quantized(q, x)
    assert torch.isnan(q.dequantize(torch.float32)[0, :n]).all()


def test_scale_tiles_round_trip():
    s = torch.randint(0, 255, (300, 24), dtype=torch.uint8, device="cuda")
    t = ep.tile_fp4_scales(s)
    assert t.shape == (3, 6, 32, 4, 4)
    assert torch.equal(ep.untile_fp4_scales(t, 300), s)
    flat = t.flatten()
    for r, b in [(0, 0), (31, 3), (32, 4), (127, 23), (128, 7), (299, 12)]:
        at = (r // 128 * 6 + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
        assert flat[at] == s[r, b]


def make_ids(T, E, K, seed, drop=0.1):
    g = gen(seed)
    ids = torch.rand((T, E), device="cuda", generator=g).topk(K, dim=1).indices.to(torch.int32)
    ids[torch.rand((T, K), device="cuda", generator=g) < drop] = -1
    return ids


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("layout,R", [("strided", 2), ("packed", 2), ("strided", 1)])
@pytest.mark.parametrize("T,N", [(1, 1), (13, 16), (301, 301), (1000, 1003)])
@pytest.mark.parametrize("onepass", ["1", "0"])
def test_dispatch_fp4(fmt, layout, R, T, N, onepass, monkeypatch):
    """One kernel, with and without its grid barrier (T * K above 2048), or kernel after kernel."""
    monkeypatch.setenv("EP_DISPATCH_ONEPASS", onepass)
    D, E, K = 1152 if T == 301 else 384, 8, 3
    buf = ep.Buffer(N, D, E, R, K, layout=layout)
    ids = make_ids(T, E, K, T)
    x = torch.randn((T, D), device="cuda", generator=gen(2)).bfloat16()
    scores = torch.rand((T, K), device="cuda", generator=gen(3))
    plain = buf.dispatch(x, scores, ids, N)
    rows = plain.recv_x.reshape(-1, D).clone()
    rs, src = plain.recv_scores.flatten().clone(), plain.recv_src.flatten().clone()
    pos = plain.layout.pos.flatten().long()
    pos = pos[pos >= 0]
    buf.workspace[:rows.numel() * 2] = 0
    d = buf.dispatch_fp4(x, scores, ids, N, format=fmt)
    assert torch.equal(d.layout.pos.flatten().long()[d.layout.pos.flatten() >= 0], pos)
    assert d.recv_x.rows == R * ep.ep_pad_tokens(N) * K
    got_scales = ep.untile_fp4_scales(d.recv_x.scales, d.recv_x.rows)[pos].cpu()
    codes, scale = F4.quantize(rows[pos], fmt)
    assert torch.equal(got_scales, scale)
    assert torch.equal(F4.unpack(d.recv_x.codes[pos]), codes)
    assert torch.equal(d.recv_scores.flatten()[pos], rs[pos])
    assert torch.equal(d.recv_src.flatten()[pos], src[pos])
    assert buf.device_error() == 0
    buf.close()


def test_dispatch_fp4_leaves_other_rows():
    T, D, E, K = 20, 256, 4, 2
    buf = ep.Buffer(T, D, E, 1, K)
    ids = make_ids(T, E, K, 5, drop=0.4)
    x = torch.randn((T, D), device="cuda").bfloat16()
    rows = buf.R * T * K
    q = ep.FP4(torch.full((rows, D // 2), 0xA5, dtype=torch.uint8, device="cuda"),
               torch.full((1, D // 128, 32, 4, 4), 0x5A, dtype=torch.uint8, device="cuda"), "mx")
    ep.ep_dispatch_fp4(buf.handle, x, torch.ones((T, K), device="cuda"), ids, T, T, q)
    used = torch.zeros(rows, dtype=torch.bool)
    n = int((ids >= 0).sum())
    used[:n] = True
    assert (q.codes[~used] == 0xA5).all()
    assert (ep.untile_fp4_scales(q.scales, 128)[n:] == 0x5A).all()
    assert not (q.codes[used] == 0xA5).all()


class Case:
    """Receive rows and weights in 4 bits, and what they stand for in 64 bits on the GPU."""

    def __init__(self, T, D, E, K, fmt, R=1, layout="packed", seed=0, drop=0.1, ids=None):
        self.fmt = fmt
        self.buf = ep.Buffer(T, D, E, R, K, layout=layout)
        self.ids = make_ids(T, E, K, seed, drop) if ids is None else ids
        g = gen(seed + 1)
        x = torch.randn((T, D), device="cuda", generator=g).bfloat16()
        self.d = self.buf.dispatch_fp4(x, torch.ones((T, K), device="cuda"), self.ids, T, format=fmt)
        self.x = self.values(self.d.recv_x)
        lay = self.d.layout
        self.spans = [(e, int(lay.expert_offset[e]), int(lay.tokens_per_expert[e])) for e in range(E)]
        self.spans = [s for s in self.spans if s[2]]
        self.g = g

    def values(self, q):
        sc = ep.untile_fp4_scales(q.scales, q.rows)
        v = F4.values(F4.unpack(q.codes.reshape(q.rows, -1)), sc, q.format)
        v = v.cuda().view(*q.codes.shape[:-1], -1)
        if q.tensor_scale is not None:
            v *= q.tensor_scale.double().view(*q.codes.shape[:-2], 1, 1)
        return v

    def weights(self, E, rows, cols, tensor_scale=False):
        codes, sc = F4.random_fp4(self.g, (E, rows), cols, self.fmt, cols ** -0.5)
        ts = None
        if tensor_scale:
            ts = torch.rand(E, device="cuda", generator=self.g) + 0.5
        w = ep.FP4(codes, ep.tile_fp4_scales(sc), self.fmt, ts)
        return w, self.values(w)


def product_bound(x, w):
    """n 2^-23 sum |x w|: any order of n fp32 additions that may cut instead of rounding."""
    return (x.abs() @ w.abs().mT) * (x.shape[-1] * 2.0 ** -23)


BF16 = 2.0 ** -8    # half a step of bf16, relative


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kernel", ["1", "2"])
@pytest.mark.parametrize("T,D,F,E,K,R,layout", [
    (1, 128, 256, 1, 1, 1, "packed"),
    (5, 256, 256, 4, 2, 2, "strided"),
    (130, 384, 512, 3, 1, 1, "packed"),
    (301, 1024, 256, 5, 3, 1, "packed"),
    (700, 640, 768, 2, 2, 2, "strided"),
])
def test_gemm(fmt, kernel, T, D, F, E, K, R, layout, monkeypatch):
    monkeypatch.setenv("EP_GEMM_KERNEL", kernel)
    c = Case(T, D, E, K, fmt, R, layout, seed=T)
    w, wv = c.weights(E, F, D, tensor_scale=fmt == "nv")
    n = c.d.recv_x.rows
    y = torch.full((n, F), 7.0, dtype=torch.bfloat16, device="cuda")
    out = c.buf.expert_gemm_fp4(c.d.recv_x, w, y)
    assert out is y
    touched = torch.zeros(n, dtype=torch.bool, device="cuda")
    for e, lo, m in c.spans:
        x = c.x[lo:lo + m]
        want = x @ wv[e].T
        # One more rounding: the fp32 product with the tensor scale.
        bound = product_bound(x, wv[e]) + (BF16 + 2.0 ** -23) * want.abs()
        assert ((y[lo:lo + m].double() - want).abs() <= bound).all(), (e, m)
        touched[lo:lo + m] = True
    assert (y[~touched] == 7.0).all()
    assert c.buf.device_error() == 0
    c.buf.close()


def act64(g, act):
    if act == "silu":
        return g * torch.special.expit(g)
    v = 2 * (2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)
    return g * torch.special.expit(v)


def glu_bound(x, wg, wu, g, u, act):
    """How far act(g) u may be off: the sums' bounds through |act'| <= 1.13 and |act| <= |g|, and
    2^-18 for the activation's own arithmetic (a few ulp of fp32, |g| well below 32)."""
    return (1.13 * product_bound(x, wg) * u.abs() + g.abs() * product_bound(x, wu)
            + 1.13 * product_bound(x, wg) * product_bound(x, wu) + 2.0 ** -18 * (g * u).abs())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kernel", ["1", "2"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,D,F,E,K", [(1, 128, 128, 1, 1), (130, 384, 256, 3, 1),
                                       (301, 512, 384, 5, 3), (600, 256, 128, 2, 2)])
def test_glu(fmt, kernel, act, T, D, F, E, K, monkeypatch):
    monkeypatch.setenv("EP_GEMM_KERNEL", kernel)
    c = Case(T, D, E, K, fmt, seed=T)
    w, wv = c.weights(E, 2 * F, D, tensor_scale=fmt == "nv")
    h = c.buf.expert_glu_fp4(c.d.recv_x, w, act)
    q = c.buf.expert_glu_fp4(c.d.recv_x, w, act, quantize=True)
    assert q.format == fmt and q.cols == F
    qv = c.values(q)
    codes, scales = q.codes, ep.untile_fp4_scales(q.scales, q.rows)
    for e, lo, m in c.spans:
        x = c.x[lo:lo + m]
        g, u = x @ wv[e][:F].T, x @ wv[e][F:].T
        want = act64(g, act) * u
        bound = glu_bound(x, wv[e][:F], wv[e][F:], g, u, act)
        assert ((h[lo:lo + m].double() - want).abs() <= bound + BF16 * want.abs()).all()
        # Quantised: the block's scale is that of an amax within the bound, and each element the
        # nearest of its grid to a number within the bound.
        sc = scales[lo:lo + m].long().cpu()
        wb = want.cpu().unflatten(-1, (-1, F4.BLOCK[fmt]))
        bb = bound.cpu().unflatten(-1, (-1, F4.BLOCK[fmt]))
        lo_c = F4.quantize((wb.abs() - bb).clamp(min=0).flatten(-2), fmt)[1].long()
        hi_c = F4.quantize((wb.abs() + bb).flatten(-2), fmt)[1].long()
        assert ((sc >= lo_c) & (sc <= hi_c)).all()
        unit = F4.values(torch.full((m, F), 2), sc, fmt).unflatten(-1, (-1, F4.BLOCK[fmt]))
        got = qv[lo:lo + m].cpu().unflatten(-1, (-1, F4.BLOCK[fmt])) / unit
        near = (wb / unit).clamp(-6, 6)
        slack = bb / unit
        # Half the step of the binade: 0.25 below 2, 0.5 below 4, 1 above; an element right at a
        # binade's border may round by the wider one.
        a = near.abs() + slack
        half = torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, 1.0))
        assert ((got - near).abs() <= half + slack).all()
    assert codes.shape == (q.rows, F // 2)
    assert c.buf.device_error() == 0
    c.buf.close()


@pytest.mark.parametrize("fmt", FORMATS)
def test_ffn(fmt):
    """The block is its two products, with h as the first one leaves it."""
    T, D, F, E, K = 257, 512, 256, 6, 2
    c = Case(T, D, E, K, fmt, seed=9)
    w1, _ = c.weights(E, 2 * F, D, tensor_scale=fmt == "nv")
    w2, w2v = c.weights(E, D, F, tensor_scale=fmt == "nv")
    hs = torch.tensor([0.37], device="cuda") if fmt == "nv" else None
    y = c.buf.expert_ffn_fp4(c.d.recv_x, w1, w2, "gelu", h_scale=hs)
    h = c.buf.expert_glu_fp4(c.d.recv_x, w1, "gelu", quantize=True, h_scale=hs)
    hv = c.values(h)
    for e, lo, m in c.spans:
        want = hv[lo:lo + m] @ w2v[e].T
        bound = product_bound(hv[lo:lo + m], w2v[e]) + (BF16 + 2.0 ** -22) * want.abs()
        assert ((y[lo:lo + m].double() - want).abs() <= bound).all()
    out = c.buf.combine(y, torch.rand((T, K), device="cuda"))
    assert torch.isfinite(out).all()
    assert c.buf.device_error() == 0
    c.buf.close()


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_block_reaches_its_own_row(fmt):
    T, D, F, E = 200, 256, 128, 2
    x = torch.randn((T, D), device="cuda", generator=gen(4)).bfloat16()
    x[17, 100] = float("nan")
    x[90, 3] = float("inf")
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    ids[150:] = 1
    buf = ep.Buffer(T, D, E, 1, 1, layout="packed")
    c, sc = F4.random_fp4(gen(5), (E, F), D, fmt)
    w = ep.FP4(c, ep.tile_fp4_scales(sc), fmt)
    y = buf.expert_gemm_fp4(buf.dispatch_fp4(x, torch.ones((T, 1), device="cuda"), ids,
                                             format=fmt).recv_x, w)
    bad = torch.isnan(y[:T]).all(1)
    assert bad.nonzero().flatten().tolist() == [17, 90]
    assert torch.isfinite(y[:T][~bad]).all()
    buf.close()


def test_capture_and_replay():
    """A step in a graph, replayed with new tokens and routing in the same buffers."""
    T, D, F, E, K = 64, 256, 128, 4, 2
    buf = ep.Buffer(T, D, E, 1, K, layout="packed")
    g = gen(6)
    ws = []
    for rows, cols in ((2 * F, D), (D, F)):
        c, sc = F4.random_fp4(g, (E, rows), cols, "nv", cols ** -0.5)
        ws.append(ep.FP4(c, ep.tile_fp4_scales(sc), "nv"))
    x = torch.randn((T, D), device="cuda", generator=g).bfloat16()
    ids, scores = make_ids(T, E, K, 7), torch.rand((T, K), device="cuda")

    def step():
        d = buf.dispatch_fp4(x, scores, ids)
        return buf.combine(buf.expert_ffn_fp4(d.recv_x, *ws), scores)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (11, 12):
        x.copy_(torch.randn((T, D), device="cuda", generator=g))
        ids.copy_(make_ids(T, E, K, seed, drop=0.5))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, step())
    assert buf.device_error() == 0
    del graph
    buf.close()


def test_empty_step():
    buf = ep.Buffer(8, 256, 4, 1, 2, layout="packed")
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    d = buf.dispatch_fp4(x, torch.empty((0, 2), device="cuda"),
                         torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    c, sc = F4.random_fp4(gen(1), (4, 128), 256, "nv")
    y = buf.expert_gemm_fp4(d.recv_x, ep.FP4(c, ep.tile_fp4_scales(sc), "nv"))
    assert y.shape == (0, 128)
    q = ep.quantize_fp4(x, "mx")
    assert q.dequantize().shape == (0, 256)
    buf.close()


def test_refusals():
    T, D, E, K = 8, 256, 4, 2
    buf = ep.Buffer(T, D, E, 1, K, layout="packed")
    x = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    scores, ids = torch.ones((T, K), device="cuda"), make_ids(T, E, K, 1)
    c, sc = F4.random_fp4(gen(1), (E, 128), D, "nv")
    w = ep.FP4(c, ep.tile_fp4_scales(sc), "nv")
    q = ep.quantize_fp4(torch.zeros((T * K, D), dtype=torch.bfloat16, device="cuda"), "nv")
    with pytest.raises(ep.EpError) as e:                      # no layout yet
        ep.ep_expert_gemm_fp4(buf.handle, q, w, D, 128,
                              torch.empty((T * K, 128), dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == ep._abi.EP_ERR_NO_LAYOUT
    with pytest.raises(ep.EpError) as e:
        buf.dispatch_fp4(x, scores, ids, T + 1)
    assert e.value.status == ep._abi.EP_ERR_CAPACITY
    with pytest.raises(ep.EpError):
        buf.dispatch_fp4(x, scores, ids, T - 1)
    with pytest.raises(ValueError, match="format"):
        buf.dispatch_fp4(x, scores, ids, format="int4")
    with pytest.raises(ValueError, match="x, scores and ids"):
        buf.dispatch_fp4(x, scores[:4], ids)
    with pytest.raises(ValueError, match="tensor_scale"):
        buf.dispatch_fp4(x, scores, ids, format="mx", tensor_scale=torch.ones(1, device="cuda"))
    rows = buf.dispatch_fp4(x, scores, ids, format="mx").recv_x
    with pytest.raises(ValueError, match="mx"):
        buf.expert_gemm_fp4(rows, w)                          # one format only
    rows = buf.dispatch_fp4(x, scores, ids).recv_x
    with pytest.raises(TypeError):
        buf.expert_gemm_fp4(rows, c)
    with pytest.raises(TypeError):
        buf.expert_gemm_fp4(x, w)
    with pytest.raises(ValueError, match="gate and up"):
        buf.expert_glu_fp4(rows, w)                           # 128 rows: no gate and up of 128 each
    c2, sc2 = F4.random_fp4(gen(2), (E, 256), D, "nv")
    wg = ep.FP4(c2, ep.tile_fp4_scales(sc2), "nv")
    with pytest.raises(ValueError, match="w_down"):
        buf.expert_ffn_fp4(rows, wg, w)                       # w_down takes 256 columns, h has 128
    with pytest.raises(ValueError, match="act"):
        buf.expert_glu_fp4(rows, wg, act="relu")
    small = ep.quantize_fp4(torch.zeros((4, D), dtype=torch.bfloat16, device="cuda"), "nv")
    with pytest.raises(ValueError, match="receive layout"):
        buf.expert_gemm_fp4(small, w)
    with pytest.raises(ValueError, match="contiguous"):
        ep.quantize_fp4(torch.zeros((4, 2 * D), dtype=torch.bfloat16, device="cuda")[:, :D])
    f32 = ep.Buffer(T, D, E, 1, K, dtype=torch.float32)
    with pytest.raises(ep.EpError) as e:
        f32.dispatch_fp4(x, scores, ids)
    assert e.value.status == ep._abi.EP_ERR_INVALID_ARG
    odd = ep.Buffer(T, 192, E, 1, K)
    with pytest.raises(ValueError, match="128"):
        odd.dispatch_fp4(x[:, :192].contiguous(), scores, ids)
    with pytest.raises(ValueError, match="changed"):
        q.codes.resize_(1, 1)
        q.dequantize()
    for b in (buf, f32, odd):
        b.close()


def test_routed_step_together():
    """As they are used: the router, the quantising dispatch, the experts in 4 bits, combine, and the
    router's gradient; and the layer for a few tokens on the same weights, which keeps x and h in
    bf16's precision, within what quantising them costs."""
    T, D, F, E, K = 48, 512, 256, 8, 2
    g = gen(21)
    buf = ep.Buffer(T, D, E, 1, K, layout="packed")
    ws = [ep.quantize_fp4((torch.randn((E, r, c), device="cuda", generator=g) * c ** -0.5).bfloat16(),
                          "nv", torch.full((E,), 2.0 ** -8, device="cuda"))
          for r, c in ((2 * F, D), (D, F))]
    x = torch.randn((T, D), device="cuda", generator=g).bfloat16()
    logits = torch.randn((T, E), device="cuda", generator=g)
    select = logits.clone()
    select[40:] = -torch.inf                       # padding
    ids, scores = ep.route(logits, K, "sigmoid", select=select)
    d = buf.dispatch_fp4(x, scores, ids)
    y = buf.expert_ffn_fp4(d.recv_x, *ws)
    out = buf.combine(y, scores)
    _, grad_scores = buf.combine_backward(torch.randn_like(out), y, scores)
    grad = ep.route_backward(grad_scores, logits, ids, "sigmoid")
    assert (out[40:] == 0).all() and (grad[40:] == 0).all() and torch.isfinite(grad).all()
    few = buf.moe_layer(x, scores, ids, *ws)
    assert (few[40:] == 0).all()
    # An element of e2m1 with a scale that fits its block is off by at most 1/12 of the block's
    # largest, 0.04 in the root mean square of normal ones; two such roundings and the gate's slope
    # keep the result within a quarter.
    off = (few.float() - out.float()).norm() / few.float().norm()
    assert 0.01 < off < 0.25
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids2, scores2 = ep.route(logits, K, "sigmoid", select=select, stream=s)
    d2 = buf.dispatch_fp4(x, scores2, ids2, stream=s)
    out2 = buf.combine(buf.expert_ffn_fp4(d2.recv_x, *ws, stream=s), scores2, stream=s)
    s.synchronize()
    assert torch.equal(out, out2)
    assert buf.device_error() == 0
    buf.close()


@pytest.mark.parametrize("offset", [8, 16])
def test_quantize_unaligned_to_32_bytes(offset):
    """A matrix at 16 bytes from a 32-byte boundary (offset 8 elements): both ways of reading."""
    flat = torch.randn(40 * 256 + 16, device="cuda", generator=gen(3)).bfloat16()
    x = flat[offset:offset + 40 * 256].view(40, 256)
    assert_quantized(ep.quantize_fp4(x, "nv"), x)
    q = ep.quantize_fp4(x, "mx")
    out = flat.clone()[offset:offset + 40 * 256].view(40, 256)
    ep.ep_dequantize_fp4(q, out)
    assert torch.equal(out, q.dequantize())


@pytest.mark.parametrize("E,rows", [(5, 1999), (2500, 7)])
def test_quantize_many_rows(E, rows):
    """More rows than warps at once, so that a warp goes from matrix to matrix, or over many."""
    g = gen(4)
    x = torch.randn((E, rows, 512), device="cuda", generator=g).bfloat16()
    ts = 0.001 * (1 + torch.rand(E, device="cuda", generator=g))
    q = ep.quantize_fp4(x, "nv", ts)
    scales = ep.untile_fp4_scales(q.scales, E * rows).view(E, rows, -1)
    for e in (0, 1, E // 2, E - 1):
        codes, scale = F4.quantize(x[e], "nv", float(ts[e].double()))
        assert torch.equal(scales[e].cpu(), scale)
        assert torch.equal(F4.unpack(q.codes[e]), codes)
        want = F4.values(codes, scale, "nv", 1.0).float() * ts[e].cpu()
        assert torch.equal(q.dequantize(torch.float32)[e].cpu(), want)
    # A matrix by itself is quantised as in the batch, its rows' other warps and lanes apart.
    for e in range(0, E, 97):
        alone = ep.quantize_fp4(x[e], "nv", ts[e:e + 1])
        assert torch.equal(alone.codes, q.codes[e])
        assert torch.equal(alone.dequantize(), q.dequantize()[e])


def test_quantize_a_matrix_of_zeros():
    """Scaled by its own largest magnitude, 0: scales and products of zeros, not NaN."""
    x = torch.randn((3, 128, 256), device="cuda", generator=gen(5)).bfloat16()
    x[1] = 0
    ts = x.abs().amax((1, 2)).float() / (6 * 448)
    q = ep.quantize_fp4(x, "nv", ts)
    assert (ep.untile_fp4_scales(q.scales, 384)[128:256] == 0).all()
    assert (q.dequantize() == 0)[1].all()
    assert torch.isfinite(q.dequantize()).all()


@pytest.mark.parametrize("T,D,E,K", [(2500, 1024, 8, 1), (1500, 640, 4, 2), (900, 512, 24, 5),
                                     (400, 256, 1024, 8), (300, 384, 64, 20)])
def test_dispatch_fp4_with_a_barrier(T, D, E, K):
    """Calls above 2048 pairs: tokens that wait in shared memory and others, few and many experts,
    also captured and replayed on other ids."""
    buf = ep.Buffer(T, D, E, 1, K)
    x = torch.randn((T, D), device="cuda", generator=gen(6)).bfloat16()
    scores = torch.rand((T, K), device="cuda", generator=gen(7))
    ts = torch.tensor([0.0021], device="cuda")
    whole = ep.quantize_fp4(x, "nv", ts)
    token_scales = ep.untile_fp4_scales(whole.scales, T)
    ids = make_ids(T, E, K, 8)

    def check(d):
        pos = d.layout.pos.flatten().long()
        src = torch.arange(T * K, device="cuda")[pos >= 0]
        pos = pos[pos >= 0]
        assert torch.equal(pos.sort().values, torch.arange(len(pos), device="cuda"))
        by_expert = ids.flatten().long()[src]
        order = by_expert.sort(stable=True).indices
        assert torch.equal(pos[order], torch.arange(len(pos), device="cuda"))
        assert torch.equal(d.recv_x.codes[pos], whole.codes[src // K])
        assert torch.equal(ep.untile_fp4_scales(d.recv_x.scales, d.recv_x.rows)[pos],
                           token_scales[src // K])
        assert torch.equal(d.recv_scores.flatten()[pos], scores.flatten()[src])
        assert torch.equal(d.recv_src.flatten()[pos].long(), src)

    check(buf.dispatch_fp4(x, scores, ids, tensor_scale=ts))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d = buf.dispatch_fp4(x, scores, ids, tensor_scale=ts)
    for seed in (9, 10):
        ids.copy_(make_ids(T, E, K, seed, drop=0.3))
        graph.replay()
        check(d)
    del graph
    assert buf.device_error() == 0
    buf.close()
