"""4-bit products of rows in which one element of a block dominates.

x is multiplied as x' = hi + lo, two 8-bit floating-point terms of a block of 128 scaled
values. An element far below the block's largest, M, is off by at most 2^-k M, so a result may
be off by sum |w| 2^-k M over such elements: nothing where the weight is zero, however large
zero point and code are. (k: BITS below; where |x| >= 2^-EXACT M, x' = x.)

The fp32 sums are of (code - zero) x' in parts, code x' and zero x': a group of G such terms
and din / G groups, within 2 (G + din / G) 2^-24 sum s (code + zero) |x|. One rounding to bf16
adds 2^-8 of the result.
"""
import pytest
import torch

import combine_topk_ids_expert_gb300 as ep
from test_expert_ffn_gpu import Case, products
from test_expert_w4_gpu import dequantised, weights

pytestmark = pytest.mark.gpu

F64 = torch.float64
EXACT, BITS = 13, 21
ROWS = [2, 7, 24]      # taken 4, 8 and 16 at a time


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", ROWS)
def test_weights_of_zero_leave_nothing(rows, group):
    # 255 and 0.2: x' of 0.2 has 9 fractional bits, and sums of 15 x' stay under 2^13, so all
    # of them are exact in fp32, and so are scales of powers of two.
    c = Case(91, rows, 1, 1, 1)
    din, dout = 512, 144
    x = c.out(din)
    x[:] = 0.2
    x[:, 7::128] = 255.0
    x[~c.used] = float("nan")
    z = torch.randint(0, 16, (1, dout, din // group), dtype=torch.uint8, device="cuda",
                      generator=c.gen)
    q = z.repeat_interleave(group, 2)
    s = torch.exp2(torch.randint(-9, 3, z.shape, device="cuda", generator=c.gen).float())
    w = ep.W4((q[..., 0::2] | (q[..., 1::2] << 4)).contiguous(), s, z)
    y = c.buf.expert_gemv_w4(x, w, c.out(dout))
    assert bool((y[c.used] == 0.0).all())
    # One weight that is not zero, at each place: that product alone.
    at = 7 + 128 * 2
    codes = w.codes.clone()
    low = codes[:, :, at // 2] & 15
    codes[:, :, at // 2] = low | ((((z[..., at // group] + 5) % 16)) << 4)
    y = c.buf.expert_gemv_w4(x, ep.W4(codes, s, z), c.out(dout))
    zd = z[0, :, at // group].to(F64)
    want = ((zd + 5) % 16 - zd) * s[0, :, at // group].to(F64) * 255.0
    assert torch.equal(y[c.used].to(F64), want.bfloat16().to(F64).expand(int(c.used.sum()), dout))
    c.done()


@pytest.mark.parametrize("zeros,scale", [(True, "f32"), (False, "bf16")])
@pytest.mark.parametrize("dominant", [0, 6, 9, 12, 15])
@pytest.mark.parametrize("rows", ROWS)
def test_the_others_keep_their_bits(rows, dominant, zeros, scale):
    # The dominant element's weights are zero: what is left is the others' sum.
    c = Case(92, rows, 1, 1, 1)
    din, dout, group = 128, 272, 32
    x = c.recv(din)
    x[:, 33] = x[:, 33].sign() * 2.0 ** dominant
    w = weights(c, dout, din, group, zeros, scale)
    z = torch.full_like(w.scales, 8, dtype=torch.uint8) if w.zeros is None else w.zeros
    w.codes[:, :, 16] = (w.codes[:, :, 16] & 15) | (z[..., 1] << 4)
    d = dequantised(w)
    assert bool((d[:, :, 33] == 0.0).all())
    y = c.buf.expert_gemv_w4(x, w, c.out(dout))
    ref, _ = products(c, x, d)
    big = x.to(F64).abs().amax(1, keepdim=True).expand_as(x)
    below = torch.where(x.to(F64).abs() >= big * 2.0 ** -EXACT, 0.0, big)
    _, off = products(c, torch.nan_to_num(below), d)
    parts = w.scales.to(F64).abs() * z.to(F64)
    _, m = products(c, x, d.abs() + 2 * parts.repeat_interleave(group, 2))
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -BITS * off + 2.0 * (group + din // group) * 2.0 ** -24 * m
    c.check_rows(y, ref, tol + 1e-38)
    c.done()
