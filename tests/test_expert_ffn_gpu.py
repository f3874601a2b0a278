"""The experts' gated feed-forward block and its gradients against plain 64-bit products.

Every product sums K exact bf16 products in fp32 in the tensor cores' order: within
2 K 2^-24 sum|a b| of the exact sum. One rounding to bf16 adds 2^-8 of the result
(half an ulp is 2^-9; the other half covers what the fp32 steps around it are off by).
The activation's __expf and __fdividef are off by at most (2 + 1.2 |v|) + 2 ulp of
fp32, under 2^-16 of the sigmoid for |v| < 50, and the slope p + g v' p (1 - p) by that
of each of its terms (1 - p by 2^-23 more). Bounds below add these terms.

Receive rows of no expert hold NaNs throughout: none may reach a result, and outputs
there keep their contents.
"""
import math

import pytest
import torch

import combine_topk_ids_expert_gb300 as ep
import workloads as W
from gpu_util import to_dev

pytestmark = pytest.mark.gpu

F64 = torch.float64
SENTINEL = 0x7FC1


def act_ref(g, act):
    """act(g), its slope and the sizes of the slope's terms, in 64 bits."""
    c = 2 * math.sqrt(2 / math.pi)
    v = g if act == "silu" else c * (g + 0.044715 * g ** 3)
    dv = torch.ones_like(g) if act == "silu" else c * (1 + 3 * 0.044715 * g ** 2)
    p, q = torch.sigmoid(v), torch.sigmoid(-v)
    return g * p, p + g * dv * p * q, p + (g * dv * p).abs() * (q + 2.0 ** -6)


class Case:
    """A buffer with a layout, receive rows in it and the experts' row ranges."""

    def __init__(self, seed, T, E, K, R, routing="uniform", layout="strided", drop=0.0, D=64):
        ids, _ = W.routing(seed, T, E, K, routing, "sigmoid_norm")
        ids = torch.from_numpy(ids).cuda()
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        if drop:
            ids[torch.rand(ids.shape, generator=self.gen, device="cuda") < drop] = -1
        self.buf = ep.Buffer(max(T, 1), D, E, R, K, dtype=torch.bfloat16, layout=layout)
        self.ids = ids
        lay = self.buf.dispatch_layout(ids, T)
        self.E, self.rows = E, R * lay.rank_stride
        off, cnt = lay.expert_offset.tolist(), lay.tokens_per_expert.tolist()
        self.spans = [(e, off[e], off[e] + cnt[e]) for e in range(E) if cnt[e]]
        self.used = torch.zeros(self.rows, dtype=torch.bool, device="cuda")
        for _, lo, hi in self.spans:
            self.used[lo:hi] = True

    def randn(self, *shape, std=1.0):
        t = torch.randn(shape, generator=self.gen, device="cuda") * std
        return t.to(torch.bfloat16)

    def recv(self, width, std=1.0):
        t = self.randn(self.rows, width, std=std)
        t[~self.used] = float("nan")
        return t

    def out(self, width):
        return torch.full((self.rows, width), SENTINEL, dtype=torch.int16,
                          device="cuda").view(torch.bfloat16)

    def check_rows(self, got, ref, tol):
        """got within tol of ref on the experts' rows, untouched elsewhere."""
        assert bool((got.view(torch.int16)[~self.used] == SENTINEL).all()), "rows of no expert"
        bad = (got.to(F64)[self.used] - ref[self.used]).abs() > tol[self.used]
        assert not bool(bad.any()), f"{int(bad.sum())} outside the bound"

    def done(self):
        torch.cuda.synchronize()
        assert self.buf.device_error() == 0
        self.buf.close()


def products(c, a, w, transpose=True):
    """(exact rows a W_e^T (or a W_e), sum |a w|) in 64 bits."""
    n = w.shape[1] if transpose else w.shape[2]
    y = torch.zeros((c.rows, n), dtype=F64, device="cuda")
    m = torch.zeros_like(y)
    for e, lo, hi in c.spans:
        we = w[e].to(F64).T if transpose else w[e].to(F64)
        y[lo:hi] = a[lo:hi].to(F64) @ we
        m[lo:hi] = a[lo:hi].to(F64).abs() @ we.abs()
    return y, m


def sum_tol(k, m):
    return 2.0 * k * 2.0 ** -24 * m


CASES = {
    # name: (seed, T, E, K, R, routing, layout, drop, din, dff, dout)
    "small":        (1, 37, 8, 2, 2, "uniform", "strided", 0.0, 64, 128, 128),
    "one_token":    (2, 1, 4, 1, 1, "uniform", "strided", 0.0, 128, 128, 256),
    "zipf":         (3, 300, 16, 4, 4, "zipf", "strided", 0.0, 256, 384, 256),
    "packed_drop":  (4, 333, 16, 4, 4, "zipf", "packed", 0.3, 192, 256, 384),
    "many_empty":   (5, 13, 256, 8, 8, "uniform", "packed", 0.0, 128, 128, 256),
    "one_expert":   (6, 777, 1, 1, 1, "uniform", "strided", 0.0, 320, 512, 256),
    "wide":         (7, 700, 3, 2, 1, "zipf", "strided", 0.1, 1024, 640, 1152),
    "e1024":        (8, 300, 1024, 8, 64, "uniform", "strided", 0.0, 64, 128, 128),
    "all_dropped":  (9, 20, 4, 2, 1, "uniform", "strided", 1.0, 128, 128, 128),
}


@pytest.fixture(params=["0", "1", "2"])
def kind(request, monkeypatch):
    """Tiles as the sizes choose them, of 128 rows on one SM, and of 256 on an SM pair where
    the sizes allow."""
    monkeypatch.setenv("EP_GEMM_KERNEL", request.param)
    return request.param


def case(name):
    seed, T, E, K, R, routing, layout, drop, din, dff, dout = CASES[name]
    return Case(seed, T, E, K, R, routing, layout, drop), din, dff, dout


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_glu(kind, name, act):
    c, din, dff, _ = case(name)
    x, w = c.recv(din), c.randn(c.E, 2 * dff, din, std=2.0 * din ** -0.5)
    gate_up, h = c.out(2 * dff), c.out(dff)
    c.buf.expert_glu(x, w, act, gate_up, h)
    again = c.buf.expert_glu(x, w, act, h=c.out(dff))
    gu, m = products(c, x, w)
    d = sum_tol(din, m)
    c.check_rows(gate_up, gu, 2.0 ** -8 * gu.abs() + d + 1e-38)
    g, u = gu[:, :dff], gu[:, dff:]
    a, _, _ = act_ref(g, act)
    dg, du = d[:, :dff], d[:, dff:]
    tol = (2.0 ** -8 + 2.0 ** -15) * (a * u).abs() + 1.13 * dg * (u.abs() + du) + a.abs() * du
    c.check_rows(h, a * u, tol + 1e-38)
    # Keeping the pre-activations changes nothing of h.
    assert torch.equal(h.view(torch.int16), again.view(torch.int16))
    c.done()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_glu_backward(kind, name, act):
    c, _, dff, dout = case(name)
    gy, w = c.recv(dout, 0.5), c.randn(c.E, dout, dff, std=dout ** -0.5)
    gate_up = c.recv(2 * dff, 2.0)
    got = c.out(2 * dff)
    c.buf.expert_glu_backward(gy, w, gate_up, act, got)
    gh, m = products(c, gy, w, transpose=False)
    d = sum_tol(dout, m)
    g, u = gate_up[:, :dff].to(F64), gate_up[:, dff:].to(F64)
    a, slope, size = act_ref(g, act)
    ref = torch.cat((gh * u * slope, gh * a), 1)
    tol = 2.0 ** -8 * ref.abs() + torch.cat(
        (d * (u * slope).abs() + (gh * u).abs() * size * 2.0 ** -15,
         d * a.abs() + (gh * a).abs() * 2.0 ** -15), 1)
    c.check_rows(got, ref, tol + 1e-38)
    c.done()


@pytest.mark.parametrize("name", sorted(CASES))
def test_gemm_backward_rows(kind, name):
    c, din, _, dout = case(name)
    gy, w = c.recv(dout), c.randn(c.E, dout, din, std=dout ** -0.5)
    got = c.out(din)
    gx, gw = c.buf.expert_gemm_backward(gy, None, w, want_weights=False, grad_x=got)
    assert gx is got and gw is None
    ref, m = products(c, gy, w, transpose=False)
    c.check_rows(got, ref, 2.0 ** -8 * ref.abs() + sum_tol(dout, m) + 1e-38)
    c.done()


@pytest.mark.parametrize("dtype,accumulate", [(torch.bfloat16, False), (torch.float32, False),
                                              (torch.bfloat16, True), (torch.float32, True)])
@pytest.mark.parametrize("name", sorted(CASES))
def test_gemm_backward_weights(name, dtype, accumulate):
    c, din, _, dout = case(name)
    gy, x = c.recv(dout), c.recv(din)
    before = c.randn(c.E, dout, din).to(dtype)
    got = before.clone()
    c.buf.expert_gemm_backward(gy, x, None, want_x=False, grad_weights=got, accumulate=accumulate)
    ref = torch.zeros((c.E, dout, din), dtype=F64, device="cuda")
    tol = torch.zeros_like(ref)
    for e, lo, hi in c.spans:
        a, b = gy[lo:hi].to(F64).T, x[lo:hi].to(F64)
        ref[e] = a @ b
        tol[e] = sum_tol(hi - lo, a.abs() @ b.abs())
    if accumulate:
        ref += before.to(F64)
        tol += 2.0 ** -23 * (ref.abs() + before.to(F64).abs())
    if dtype == torch.bfloat16:
        tol += 2.0 ** -8 * ref.abs()
    bad = (got.to(F64) - ref).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} outside the bound"
    c.done()


@pytest.mark.parametrize("name", ["zipf", "packed_drop", "wide"])
def test_block_is_its_parts(kind, name):
    # expert_ffn and expert_ffn_backward give what their calls give one by one.
    c, din, dff, dout = case(name)
    x, wgu = c.recv(din), c.randn(c.E, 2 * dff, din, std=din ** -0.5)
    wd, gy = c.randn(c.E, dout, dff, std=dff ** -0.5), c.recv(dout)
    y, h, gu = c.buf.expert_ffn(x, wgu, wd, save=True)
    gate_up = c.out(2 * dff)
    h1 = c.buf.expert_glu(x, wgu, "silu", gate_up)
    parts = [(y, c.buf.expert_gemm(h1, wd)), (h, h1), (gu, gate_up),
             (c.buf.expert_ffn(x, wgu, wd), y)]
    gx, gwgu, gwd = c.buf.expert_ffn_backward(gy, x, wgu, wd, gu, h)
    ggu = c.buf.expert_glu_backward(gy, wd, gu)
    gx1, gwgu1 = c.buf.expert_gemm_backward(ggu, x, wgu)
    _, gwd1 = c.buf.expert_gemm_backward(gy, h, None, want_x=False)
    parts += [(gx, gx1)]
    for a, b in parts:
        a, b = (t.reshape(c.rows, -1)[c.used].view(torch.int16) for t in (a, b))
        assert torch.equal(a, b)
    assert torch.equal(gwgu, gwgu1) and torch.equal(gwd, gwd1)
    c.done()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_against_differences(act):
    # The loss sum(grad_y * y) of the 64-bit formula, differentiated by central
    # differences along random directions, against the kernels' gradients along them.
    # The step's truncation and cancellation stay under 1e-6 of the loss's scale; the
    # kernels' bf16 roundings (saved pre-activations, h, grad g and u, the results: at
    # most four of 2^-9 in a chain) are independent over thousands of elements.
    c = Case(21, 120, 4, 2, 2, "zipf")
    din, dff, dout = 128, 256, 128
    x, wgu = c.recv(din), c.randn(c.E, 2 * dff, din, std=din ** -0.5)
    wd, gy = c.randn(c.E, dout, dff, std=dff ** -0.5), c.recv(dout)
    _, h, gu = c.buf.expert_ffn(x, wgu, wd, act, save=True)
    grads = c.buf.expert_ffn_backward(gy, x, wgu, wd, gu, h, act)

    def loss(x, wgu, wd):
        total = 0.0
        for e, lo, hi in c.spans:
            p = x[lo:hi] @ wgu[e].T
            y = (act_ref(p[:, :dff], act)[0] * p[:, dff:]) @ wd[e].T
            total += float((y * gy[lo:hi].to(F64)).sum())
        return total

    at = [t.to(F64) for t in (x, wgu, wd)]
    at[0][~c.used] = 0.0
    for i in range(3):
        d = torch.randn(at[i].shape, generator=c.gen, device="cuda", dtype=F64)
        grad = grads[i].reshape(at[i].shape).to(F64)
        if i == 0:
            d[~c.used] = 0.0
            grad = torch.where(c.used[:, None], grad, 0.0)
        eps = 1e-4
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + eps * d, at[i] - eps * d
        want = (loss(*up) - loss(*down)) / (2 * eps)
        scale = float((grad * d).norm())      # of a sum of independent terms
        assert abs(float((grad * d).sum()) - want) <= 4 * 4 * 2.0 ** -9 * scale, i
    c.done()


def test_back_to_back_runs_agree(kind):
    # Forward and backward, call behind call: every run gives the bits of the first.
    c = Case(71, 1500, 12, 4, 2, "zipf")
    din, dff, dout = 1024, 768, 1024
    x, wgu = c.recv(din), c.randn(c.E, 2 * dff, din, std=din ** -0.5)
    wd, gy = c.randn(c.E, dout, dff, std=dff ** -0.5), c.recv(dout)

    def run():
        y, h, gu = c.buf.expert_ffn(x, wgu, wd, save=True)
        gx, gwgu, gwd = c.buf.expert_ffn_backward(gy, x, wgu, wd, gu, h)
        rows = [t.reshape(c.rows, -1)[c.used] for t in (y, h, gu, gx)]
        return [t.view(torch.int16) for t in (*rows, gwgu, gwd)]

    runs = [run() for _ in range(6)]
    for r in runs[1:]:
        for a, b in zip(runs[0], r):
            assert torch.equal(a, b)
    c.done()


def test_no_rows_at_all():
    # num_tokens_per_rank 0: nothing is routed; the weights' gradient is zero.
    buf = ep.Buffer(8, 64, 4, 1, 2, dtype=torch.bfloat16)
    buf.dispatch_layout(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 0)
    def rows(w):
        return torch.empty((0, w), dtype=torch.bfloat16, device="cuda")
    gw = torch.full((4, 128, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    h = ep.ep_expert_gemm_backward
    spare = torch.empty((1, 128), dtype=torch.bfloat16, device="cuda")
    h(buf.handle, spare, spare, None, 64, 128, None, gw, accumulate=True)
    assert bool((gw == 7.0).all())
    h(buf.handle, spare, spare, None, 64, 128, None, gw)
    torch.cuda.synchronize()
    assert bool((gw == 0.0).all())
    buf.close()


def test_extreme_gates():
    # Gates far out on both sides, where e^-v overflows or vanishes, and pre-activations
    # at bf16's ends: finite where the formula is, zeros and signs as its limits.
    c = Case(31, 64, 1, 1, 1)
    dff = dout = 128
    gate = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 88.0, -88.0, 95.0, -95.0, 1e4,
                         -1e4, 1e18, -1e18], device="cuda").to(torch.bfloat16)
    gate_up = c.recv(2 * dff)
    gate_up[c.used] = gate_up[c.used].index_copy(
        1, torch.arange(14, device="cuda"), gate.expand(int(c.used.sum()), 14))
    gy = c.recv(dout)
    wd = torch.eye(dout, device="cuda", dtype=torch.bfloat16)[None].contiguous()   # grad h = gy
    for act in ("silu", "gelu"):
        got = c.out(2 * dff)
        c.buf.expert_glu_backward(gy, wd, gate_up, act, got)
        g, u, gh = (t[c.used].to(F64) for t in (gate_up[:, :dff], gate_up[:, dff:], gy))
        a, slope, size = act_ref(g, act)
        size = torch.nan_to_num(size, nan=1.0)
        slope = torch.where(g > 1e3, 1.0, torch.where(g < -1e3, 0.0, slope))
        ref = torch.cat((gh * u * slope, gh * a), 1)
        tol = 2.0 ** -8 * ref.abs() + torch.cat(((gh * u).abs() * size.clamp(max=2.0) * 2.0 ** -15,
                                                 (gh * a).abs() * 2.0 ** -13), 1) + 1e-30
        bad = ~((got[c.used].to(F64) - ref).abs() <= tol)
        assert not bool(bad.any()), (act, bad.nonzero()[:4].tolist())
    c.done()


def test_nonfinite_rows_stay_in_their_row_and_expert():
    # An infinity in one row of x or grad_y: other rows and other experts' gradients
    # are those of the clean call, bit for bit.
    c = Case(41, 100, 4, 2, 1, "zipf")
    din, dout = 128, 128
    gy, x, w = c.recv(dout), c.recv(din), c.randn(c.E, dout, din)
    gx0, gw0 = c.buf.expert_gemm_backward(gy, x, w)
    e, lo, hi = c.spans[1]
    bad = gy.clone()
    bad[hi - 1, 5] = float("inf")
    gx1, gw1 = c.buf.expert_gemm_backward(bad, x, w)
    keep = c.used.clone()
    keep[hi - 1] = False
    i16 = torch.int16
    gx0, gx1 = gx0.reshape(c.rows, -1), gx1.reshape(c.rows, -1)
    assert torch.equal(gx0[keep].view(i16), gx1[keep].view(i16))
    assert not bool(gx1[hi - 1].isfinite().any())
    others = torch.arange(c.E, device="cuda") != e
    assert torch.equal(gw0[others].view(i16), gw1[others].view(i16))
    assert torch.equal(gw0[e, torch.arange(dout) != 5].view(i16), gw1[e, torch.arange(dout) != 5].view(i16))
    assert not bool(gw1[e, 5].isfinite().any())
    c.done()


def test_graph_replay_fresh_routing(kind):
    # Captured once, forward and backward; each replay follows that replay's counts.
    T, E, K, R, din, dff = 200, 8, 2, 2, 128, 256
    buf = ep.Buffer(T, din, E, R, K, dtype=torch.bfloat16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(51)
    bf = torch.bfloat16
    x = torch.randn((T, din), generator=gen, device="cuda").to(bf)
    wgu = (torch.randn((E, 2 * dff, din), generator=gen, device="cuda") * din ** -0.5).to(bf)
    wd = (torch.randn((E, din, dff), generator=gen, device="cuda") * dff ** -0.5).to(bf)
    ids = torch.empty((T, K), dtype=torch.int32, device="cuda")
    sc = torch.empty((T, K), dtype=torch.float32, device="cuda")

    def step(stream=None):
        d = buf.dispatch(x, sc, ids, T, stream=stream)
        y, h, gu = buf.expert_ffn(d.recv_x, wgu, wd, save=True, stream=stream)
        out = buf.combine(y, sc, stream=stream)
        grads = buf.expert_ffn_backward(y, d.recv_x, wgu, wd, gu, h, stream=stream)
        return out, buf.dispatch_backward(grads[0], T, stream=stream)[0], grads[1], grads[2]

    def route(i):
        a, b = W.routing(60 + i, T, E, K, "zipf" if i % 2 else "uniform", "sigmoid_norm")
        ids.copy_(torch.from_numpy(a))
        sc.copy_(torch.from_numpy(b))

    route(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = step()
    for i in range(3):
        route(i)
        graph.replay()
        got = [t.clone() for t in held]
        for a, b in zip(got, step()):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    torch.cuda.synchronize()
    assert buf.device_error() == 0
    buf.close()


def test_other_stream(kind):
    # Launched on a stream that is not the current one: the scratch rows of the call
    # are not handed out again while its kernels run.
    c, din, dff, dout = case("wide")
    x, wgu = c.recv(din), c.randn(c.E, 2 * dff, din, std=din ** -0.5)
    wd, gy = c.randn(c.E, dout, dff, std=dff ** -0.5), c.recv(dout)
    y0, h, gu = c.buf.expert_ffn(x, wgu, wd, save=True)
    g0 = c.buf.expert_ffn_backward(gy, x, wgu, wd, gu, h)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y1 = c.buf.expert_ffn(x, wgu, wd, stream=s)
    junk = [torch.full((c.rows, dff), 5.0, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    g1 = c.buf.expert_ffn_backward(gy, x, wgu, wd, gu, h, stream=s.cuda_stream)
    junk += [torch.full((c.rows, 2 * dff), 5.0, device="cuda", dtype=torch.bfloat16)
             for _ in range(4)]
    torch.cuda.synchronize()
    flat = [t.reshape(c.rows, -1)[c.used] for t in (y0, y1, g0[0], g1[0])]
    assert torch.equal(flat[0], flat[1]) and torch.equal(flat[2], flat[3])
    assert torch.equal(g0[1], g1[1]) and torch.equal(g0[2], g1[2])
    c.done()


def test_refusals():
    c = Case(61, 16, 4, 2, 1)
    bf = torch.bfloat16
    x, w, wd = c.recv(128), c.randn(4, 256, 128), c.randn(4, 128, 128)
    with pytest.raises(ValueError, match="act"):
        c.buf.expert_glu(x, w, "relu")
    with pytest.raises(ValueError, match="w_gate_up"):
        c.buf.expert_glu(x, w[:3].contiguous())
    with pytest.raises(ValueError, match="x_recv"):
        c.buf.expert_glu(x[:-1].contiguous(), w)
    with pytest.raises(ValueError, match="w_down"):
        c.buf.expert_ffn(x, w, c.randn(4, 128, 256))
    with pytest.raises(TypeError, match="x_recv"):
        c.buf.expert_glu(x.float(), w)
    with pytest.raises(ValueError, match="contiguous"):
        c.buf.expert_glu(c.recv(256)[:, ::2], w)
    with pytest.raises(ValueError, match="accumulate"):
        c.buf.expert_gemm_backward(x, x, wd, accumulate=True)
    with pytest.raises(TypeError, match="grad_weights"):
        c.buf.expert_gemm_backward(x, x, wd, grad_weights=wd.half())

    def status(fn, *args):
        with pytest.raises(ep.EpError) as info:
            fn(*args)
        return info.value.status

    A = ep._abi
    h, gu = c.out(128), c.out(256)
    H = c.buf.handle
    assert status(ep.ep_expert_glu, H, x, w, 96, 128, 0, None, h) == A.EP_ERR_INVALID_ARG
    assert status(ep.ep_expert_glu, H, x, w, 128, 64, 0, None, h) == A.EP_ERR_INVALID_ARG
    assert status(ep.ep_expert_glu, H, x, w, 128, 128, 2, None, h) == A.EP_ERR_INVALID_ARG
    odd = torch.empty(c.rows * 128 + 8, dtype=bf, device="cuda")[1:1 + c.rows * 128].view(c.rows, 128)
    assert status(ep.ep_expert_glu, H, odd, w, 128, 128, 0, None, h) == A.EP_ERR_ALIGNMENT
    assert status(ep.ep_expert_glu, H, x, w, 2 ** 31, 128, 0, None, h) == A.EP_ERR_CAPACITY
    assert status(ep.ep_expert_glu, H, x, w, 128, 2 ** 40, 0, None, h) == A.EP_ERR_CAPACITY
    assert status(ep.ep_expert_glu_backward, H, x, wd, gu, 64, 128, 0, gu) == A.EP_ERR_INVALID_ARG
    assert status(ep.ep_expert_gemm_backward, H, x, x, wd, 128, 128) == A.EP_ERR_INVALID_ARG
    assert status(ep.ep_expert_gemm_backward, H, x, None, None, 128, 128, h) == A.EP_ERR_INVALID_ARG
    assert status(ep.ep_expert_gemm_backward, H, x, None, None, 128, 128, None,
                  wd) == A.EP_ERR_INVALID_ARG
    f32 = ep.Buffer(16, 128, 4, 1, 2, dtype=torch.float32)
    assert status(ep.ep_expert_glu, f32.handle, x, w, 128, 128, 0, None, h) == A.EP_ERR_NO_LAYOUT
    f32.dispatch_layout(c.ids, 16)
    assert status(ep.ep_expert_glu, f32.handle, x, w, 128, 128, 0, None, h) == A.EP_ERR_INVALID_ARG
    f32.close()
    c.done()
