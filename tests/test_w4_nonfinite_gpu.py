"""Infinities and NaNs in rows of the 4-bit products: with 4, 8 and 16 rows at a time, in the
plain and the gated form, and where a row of x is held in parts. They reach their own row's
results alone: there, what the formula gives (an infinity times a weight of zero is a NaN);
every other row is that of the clean call, bit for bit."""
import pytest
import torch

from test_expert_ffn_gpu import Case, act_ref
from test_expert_w4_gpu import dequantised, weights

pytestmark = pytest.mark.gpu

F64 = torch.float64
# (tokens of one expert, din, group): 4, 8, 16 rows at a time; longer than shared memory holds.
SIZES = [(2, 256, 128), (7, 320, 64), (24, 256, 32), (40, 512, 128), (9, 16384, 128), (2, 20480, 32)]


def spoilt(c, x):
    """x with an infinity, a NaN and both signs of infinity in three rows (two of them where
    there are only two), and those rows."""
    x, din = x.clone(), x.shape[1]
    lo, hi = c.spans[0][1:]
    rows = sorted({lo, (lo + hi) // 2, hi - 1})
    for i, r in enumerate(rows):
        if i % 3 == 0:
            x[r, 5] = float("inf")
        elif i % 3 == 1:
            x[r, din - 1] = float("nan")
        else:
            x[r, 2], x[r, din // 2 + 3] = float("inf"), float("-inf")
    return x, rows


def kinds(t):
    """0 finite, 1 infinite, 2 negatively so, 3 NaN"""
    return torch.where(t.isnan(), 3, torch.where(t.isinf(), torch.where(t > 0, 1, 2), 0))


def others(c, rows):
    keep = c.used.clone()
    keep[rows] = False
    return keep


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("zeros", [False, True])
def test_products(size, zeros):
    T, din, group = size
    c = Case(94, T, 1, 1, 1)
    x, w = c.recv(din), weights(c, 88, din, group, zeros, "f32")
    clean = c.buf.expert_gemv_w4(x, w, c.out(88))
    bad, rows = spoilt(c, x)
    got = c.buf.expert_gemv_w4(bad, w, c.out(88))
    keep = others(c, rows)
    assert torch.equal(got[keep].view(torch.int16), clean[keep].view(torch.int16))
    terms = bad[rows].to(F64)[:, None, :] * dequantised(w)[0][None]
    assert torch.equal(kinds(got[rows]), kinds(terms.sum(-1)))
    c.done()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_gated_block(size, act):
    T, din, group = size
    c = Case(95, T, 1, 1, 1)
    x, w = c.recv(din), weights(c, 2 * 72, din, group, True, "bf16")
    clean = c.buf.expert_glu_w4(x, w, act, c.out(72))
    bad, rows = spoilt(c, x)
    got = c.buf.expert_glu_w4(bad, w, act, c.out(72))
    keep = others(c, rows)
    assert torch.equal(got[keep].view(torch.int16), clean[keep].view(torch.int16))
    gu = (bad[rows].to(F64)[:, None, :] * dequantised(w)[0][None]).sum(-1)
    want = act_ref(gu[:, :72], act)[0] * gu[:, 72:]
    assert torch.equal(kinds(got[rows]), kinds(want))
    c.done()
