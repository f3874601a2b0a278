"""Products with 4-bit weights and group scales against plain 64-bit products.

Codes and the two terms of x are exact as fp8 and their products in fp32, so a group's
sums and the sum of the din / G scaled groups are fp32 sums, held to the bound of the
direct sum: within 2 din 2^-24 sum|w x| of the exact one. (x below 2^-9 of its block's
largest may be off by 2^-17 of that: nothing of that size among normal rows counts; the
test of extreme rows allows for it.) One rounding to bf16 adds 2^-8 of the result (half
an ulp is 2^-9; the other half covers the activation's few ulp of fp32, as for the bf16
block).
Receive rows of no expert hold NaNs: none may reach a result, and outputs there keep
their contents.
"""
import pytest
import torch

import combine_topk_ids_expert_gb300 as ep
from test_expert_ffn_gpu import Case, act_ref, products, sum_tol

pytestmark = pytest.mark.gpu

F64 = torch.float64


def weights(c, rows, din, group, zeros, scale):
    gen = c.gen
    shape = (c.E, rows, din // group)
    codes = torch.randint(0, 256, (c.E, rows, din // 2), dtype=torch.uint8, device="cuda",
                          generator=gen)
    s = (torch.rand(shape, device="cuda", generator=gen) + 0.5) * din ** -0.5 / 4
    s *= torch.where(torch.rand(shape, device="cuda", generator=gen) < 0.5, -1.0, 1.0)
    s = s.to(torch.bfloat16) if scale == "bf16" else s
    z = None
    if zeros:
        z = torch.randint(0, 16, shape, dtype=torch.uint8, device="cuda", generator=gen)
    return ep.W4(codes, s, z)


def dequantised(w):
    q = torch.stack((w.codes & 15, w.codes >> 4), -1).flatten(2).to(F64)
    z = torch.full_like(w.scales, 8, dtype=F64) if w.zeros is None else w.zeros.to(F64)
    return ((q - z.repeat_interleave(w.group, 2)) * w.scales.to(F64).repeat_interleave(w.group, 2))


CASES = {
    # name: (seed, T, E, K, R, routing, layout, drop, din, dout, group, zeros, scale)
    "one_token":   (1, 1, 8, 2, 2, "uniform", "strided", 0.0, 256, 128, 128, False, "bf16"),
    "one_expert":  (2, 1, 1, 1, 1, "uniform", "strided", 0.0, 1024, 264, 64, True, "f32"),
    "tiny":        (3, 3, 4, 1, 1, "uniform", "packed", 0.0, 32, 8, 32, True, "bf16"),
    "odd_chunks":  (4, 9, 8, 2, 2, "zipf", "strided", 0.2, 96, 72, 32, True, "f32"),
    "odd_groups":  (5, 13, 8, 2, 2, "zipf", "packed", 0.0, 832, 200, 64, False, "f32"),
    "rows_9":      (6, 9, 1, 1, 1, "uniform", "strided", 0.0, 640, 320, 128, True, "bf16"),
    "rows_many":   (7, 150, 4, 2, 1, "zipf", "strided", 0.1, 512, 136, 32, True, "bf16"),
    "rows_300":    (8, 300, 2, 1, 1, "zipf", "strided", 0.0, 256, 128, 64, False, "bf16"),
    "e256":        (9, 31, 256, 8, 8, "uniform", "strided", 0.0, 384, 256, 128, False, "bf16"),
    "e1024":       (10, 17, 1024, 8, 64, "uniform", "packed", 0.0, 128, 64, 128, True, "f32"),
    "long":        (11, 5, 3, 2, 1, "uniform", "strided", 0.0, 7168, 96, 128, False, "bf16"),
    "long_fine":   (12, 40, 3, 2, 1, "uniform", "strided", 0.0, 4128, 96, 32, True, "f32"),
    "all_dropped": (13, 6, 4, 2, 1, "uniform", "strided", 1.0, 128, 64, 64, False, "bf16"),
    "few_zipf":    (15, 40, 64, 2, 2, "zipf", "strided", 0.1, 544, 200, 32, True, "f32"),
    "few_long":    (16, 4, 8, 2, 1, "uniform", "packed", 0.0, 4224, 136, 128, True, "bf16"),
    "units_many":  (14, 24, 64, 4, 4, "uniform", "strided", 0.0, 128, 1024, 64, True, "bf16"),
}


def case(name):
    seed, T, E, K, R, routing, layout, drop, din, dout, group, zeros, scale = CASES[name]
    c = Case(seed, T, E, K, R, routing, layout, drop)
    return c, din, dout, (group, zeros, scale)


@pytest.mark.parametrize("name", sorted(CASES))
def test_gemv(name):
    c, din, dout, kind = case(name)
    x, w = c.recv(din), weights(c, dout, din, *kind)
    y = c.out(dout)
    assert c.buf.expert_gemv_w4(x, w, y) is y
    ref, m = products(c, x, dequantised(w))
    c.check_rows(y, ref, 2.0 ** -8 * ref.abs() + sum_tol(din, m) + 1e-38)
    again = c.buf.expert_gemv_w4(x, w, c.out(dout))
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    c.done()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_glu(name, act):
    c, din, dff, kind = case(name)
    x, w = c.recv(din), weights(c, 2 * dff, din, *kind)
    h = c.out(dff)
    c.buf.expert_glu_w4(x, w, act, h)
    gu, m = products(c, x, dequantised(w))
    d = sum_tol(din, m)
    g, u, dg, du = gu[:, :dff], gu[:, dff:], d[:, :dff], d[:, dff:]
    a, _, _ = act_ref(g, act)
    tol = (2.0 ** -8 + 2.0 ** -15) * (a * u).abs() + 1.13 * dg * (u.abs() + du) + a.abs() * du
    c.check_rows(h, a * u, tol + 1e-38)
    c.done()


@pytest.mark.parametrize("name", ["few_long", "odd_chunks", "rows_many"])
def test_rows_and_scales_at_their_least_alignment(name):
    # x 16 bytes and scales an element past what allocations give: the same bits.
    c, din, dout, kind = case(name)
    x, w = c.recv(din), weights(c, dout, din, *kind)

    def past(t, n):
        flat = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")[n:]
        return flat.copy_(t.reshape(-1)).view(t.shape)

    y = c.buf.expert_gemv_w4(x, w).reshape(c.rows, -1)
    w2 = ep.W4(w.codes, past(w.scales, 1), None if w.zeros is None else past(w.zeros, 1))
    for xs, ws in ((past(x, 8), w), (x, w2)):
        got = c.buf.expert_gemv_w4(xs, ws).reshape(c.rows, -1)
        assert torch.equal(got[c.used].view(torch.int16), y[c.used].view(torch.int16))
    c.done()


def test_every_code_and_zero():
    # x picks single elements: each result is one weight, exact before its rounding.
    c = Case(20, 32, 1, 1, 1)
    x = c.out(32)
    x.copy_(torch.eye(32, device="cuda"))
    codes = torch.arange(256, device="cuda", dtype=torch.uint8).view(1, 16, 16)
    for zero in range(16):
        z = torch.full((1, 16, 1), zero, dtype=torch.uint8, device="cuda")
        s = torch.full((1, 16, 1), 0.5, device="cuda")
        y = c.buf.expert_gemv_w4(x, ep.W4(codes, s, z)).reshape(32, 16)
        want = torch.stack((codes & 15, codes >> 4), -1).flatten(2)[0].T.float() - zero
        assert torch.equal(y.float(), want * 0.5), zero
    c.done()


def test_ffn_is_its_parts_and_feeds_combine():
    c, din, dff, kind = case("odd_groups")
    c.buf.close()
    c = Case(5, 13, 8, 2, 2, "zipf", "packed", D=320)
    x, wgu = c.recv(320), weights(c, 2 * 192, 320, 64, True, "bf16")
    wd = weights(c, 320, 192, 32, False, "f32")
    y = c.buf.expert_ffn_w4(x, wgu, wd, "gelu")
    parts = c.buf.expert_gemv_w4(c.buf.expert_glu_w4(x, wgu, "gelu"), wd)
    i16 = torch.int16
    assert torch.equal(y.reshape(c.rows, -1)[c.used].view(i16),
                       parts.reshape(c.rows, -1)[c.used].view(i16))
    sc = torch.rand((13, 2), device="cuda")
    out = c.buf.combine(y, sc)
    torch.cuda.synchronize()
    assert bool(out.isfinite().all())
    c.done()


def test_back_to_back_runs_agree():
    # Long contractions over many experts, one call behind the other: the ring of codes
    # turns over while conversions, copies and products of several tiles are in flight.
    # Every run gives the bits of the first, and those are right.
    c = Case(21, 32, 96, 8, 1, "uniform", "packed")
    din, dout = 7168, 1024
    w = [weights(c, dout, din, 128, False, "bf16") for _ in range(2)]
    x = c.recv(din)
    ref, m = products(c, x, dequantised(w[0]))
    first = c.buf.expert_gemv_w4(x, w[0], c.out(dout))
    c.check_rows(first, ref, 2.0 ** -8 * ref.abs() + sum_tol(din, m) + 1e-38)
    del ref, m
    runs = [c.buf.expert_gemv_w4(x, w[i % 2], c.out(dout)) for i in range(24)]
    for i in range(0, 24, 2):
        assert torch.equal(runs[i].view(torch.int16), first.view(torch.int16)), i
        assert torch.equal(runs[i + 1].view(torch.int16), runs[1].view(torch.int16)), i
    c.done()


def test_long_contraction_in_parts():
    # x of 8 rows does not fit in shared memory: it is converted part by part, for every
    # tile again.
    c = Case(22, 11, 3, 2, 1, "zipf")
    for din, group in ((16384, 128), (11008, 32)):
        x, w = c.recv(din), weights(c, 200, din, group, True, "bf16")
        y = c.buf.expert_gemv_w4(x, w, c.out(200))
        ref, m = products(c, x, dequantised(w))
        c.check_rows(y, ref, 2.0 ** -8 * ref.abs() + sum_tol(din, m) + 1e-38)
    c.done()


def test_extreme_rows():
    # Rows at both ends of bf16's range, and rows whose elements span it: an element far
    # below its block's largest may be off by 2^-17 of that, or by 2^-136 (see the kernel),
    # which the bound allows for each element.
    c = Case(23, 6, 1, 1, 1)
    din, dout = 512, 64
    x, w = c.recv(din), weights(c, dout, din, 64, True, "f32")
    x[0] = x[0].sign() * 2.0 ** 126
    x[1] *= 2.0 ** -126
    x[2] = 0.0
    x[3] *= torch.exp2(torch.randint(-40, 40, (din,), generator=c.gen, device="cuda").float())
    x[4, 7] = 3e4
    y = c.buf.expert_gemv_w4(x, w, c.out(dout))
    d = dequantised(w)
    ref, m = products(c, x, d)
    block = x.to(F64).abs().view(c.rows, -1, 128).amax(2).repeat_interleave(128, 1)
    _, off = products(c, torch.nan_to_num(block).clamp(min=2.0 ** -119), d)
    tol = 2.0 ** -8 * ref.abs() + sum_tol(din, m) + 2.0 ** -17 * off + 1e-38
    got = y.to(F64)
    assert bool((got[2] == 0.0).all())
    c.check_rows(y, ref, tol)
    c.done()


def test_rows_do_not_depend_on_their_batch():
    # A row's result is the same whether it comes alone or among others.
    c = Case(30, 1, 1, 1, 1)
    x1, w = c.recv(512), weights(c, 128, 512, 64, True, "bf16")
    y1 = c.buf.expert_gemv_w4(x1, w).reshape(-1, 128)[:1].clone()
    c2 = Case(30, 21, 1, 1, 1)
    x2 = c2.recv(512)
    for at in (0, 7, 8, 20):
        x2[at] = x1[0]
    y2 = c2.buf.expert_gemv_w4(x2, w).reshape(-1, 128)
    for at in (0, 7, 8, 20):
        assert torch.equal(y2[at], y1[0]), at
    c.done()
    c2.done()


def test_nonfinite_rows_stay_in_their_row():
    c = Case(31, 24, 2, 1, 1)
    x, w = c.recv(256), weights(c, 64, 256, 128, False, "bf16")
    y0 = c.buf.expert_gemv_w4(x, w).reshape(c.rows, -1).clone()
    x[3, 17], x[9, 200] = float("inf"), float("nan")
    y1 = c.buf.expert_gemv_w4(x, w).reshape(c.rows, -1)
    keep = c.used.clone()
    keep[3] = keep[9] = False
    assert torch.equal(y0[keep], y1[keep])
    assert bool(y1[9].isnan().all()) and not bool(y1[3].isfinite().any())
    c.done()


def test_graph_replay_fresh_routing():
    T, E, K, R, din, dff = 9, 16, 2, 2, 256, 128
    buf = ep.Buffer(T, din, E, R, K, dtype=torch.bfloat16)
    c = Case(40, T, E, K, R)
    wgu, wd = weights(c, 2 * dff, din, 64, True, "bf16"), weights(c, din, dff, 64, True, "bf16")
    x = c.randn(T, din)
    ids = torch.empty((T, K), dtype=torch.int32, device="cuda")
    sc = torch.rand((T, K), device="cuda", generator=c.gen)

    def step():
        d = buf.dispatch(x, sc, ids, T)
        return buf.combine(buf.expert_ffn_w4(d.recv_x, wgu, wd), sc)

    def route(i):
        ids.copy_(torch.rand((T, E), generator=c.gen, device="cuda").topk(K).indices)

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
    for i in range(4):
        route(i)
        graph.replay()
        got = held.clone()
        assert torch.equal(got.view(torch.int16), step().view(torch.int16))
    torch.cuda.synchronize()
    assert buf.device_error() == 0
    buf.close()
    c.done()


def test_refusals():
    c = Case(50, 4, 2, 1, 1)
    x, w = c.recv(256), weights(c, 64, 256, 64, True, "bf16")
    with pytest.raises(TypeError, match="codes"):
        ep.W4(w.codes.float(), w.scales)
    with pytest.raises(TypeError, match="scales"):
        ep.W4(w.codes, w.scales.half())
    with pytest.raises(ValueError, match="fit"):
        ep.W4(w.codes, w.scales[:, :-1])
    with pytest.raises(ValueError, match="zeros"):
        ep.W4(w.codes, w.scales, w.zeros[:, :-1])
    with pytest.raises(ValueError, match="x_recv"):
        c.buf.expert_gemv_w4(c.recv(128), w)
    with pytest.raises(ValueError, match="w_down"):
        c.buf.expert_ffn_w4(x, w, w)
    with pytest.raises(ValueError, match="contiguous"):
        c.buf.expert_gemv_w4(x, ep.W4(w.codes[:, ::2], w.scales[:, ::2]))

    def status(fn, *args):
        with pytest.raises(ep.EpError) as info:
            fn(*args)
        return info.value.status

    A, H, y = ep._abi, c.buf.handle, c.out(64)
    g16 = ep.W4(w.codes, torch.ones((2, 64, 16), device="cuda"))
    assert status(ep.ep_expert_gemv_w4, H, x, g16, 256, 64, y) == A.EP_ERR_INVALID_ARG
    assert status(ep.ep_expert_gemv_w4, H, x, w, 224, 64, y) == A.EP_ERR_INVALID_ARG
    assert status(ep.ep_expert_gemv_w4, H, x, w, 256, 60, y) == A.EP_ERR_INVALID_ARG
    assert status(ep.ep_expert_glu_w4, H, x, w, 256, 32, 7, y) == A.EP_ERR_INVALID_ARG
    assert status(ep.ep_expert_gemv_w4, H, x, w, 256, 2 ** 31, y) == A.EP_ERR_CAPACITY
    odd = torch.empty(c.rows * 256 + 8, dtype=torch.bfloat16, device="cuda")
    odd = odd[4:4 + c.rows * 256].view(c.rows, 256)
    assert status(ep.ep_expert_gemv_w4, H, odd, w, 256, 64, y) == A.EP_ERR_ALIGNMENT
    c.done()
