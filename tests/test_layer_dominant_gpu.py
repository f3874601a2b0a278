"""What the layer for a few tokens holds of its activations. The 4-bit form: of those far below the
largest of their block, shown by weights that are zero at the large ones. On bf16 weights: all of
h."""
import pytest
import torch

import combine_topk_ids_expert_gb300 as ep
import fp4_util as F4
from test_fp4_gpu import gen
from test_moe_layer_gpu import Layer

pytestmark = pytest.mark.gpu


class Fine(Layer):
    """Layer with the bounds of eight digits."""

    def rest(self, x, h=False):
        """x: bf16 down to 2^-14 of its block's largest exact, every other element within 2^-22 of
        the largest; nv: 2^-39 of the row's largest."""
        n = F4.BLOCK[self.fmt]
        block = x.abs().unflatten(-1, (-1, n)).amax(-1, keepdim=True).expand(-1, -1, n).flatten(-2)
        rest = block * 2.0 ** -22
        if not h:
            rest = torch.where(x.abs() * 2.0 ** 14 >= block, 0.0, rest)
        if self.fmt == "nv":
            rest = torch.maximum(rest, x.abs().amax(-1, keepdim=True) * 2.0 ** -39)
        return rest

    def sums(self, x, w, h=False):
        """n 2^-23 sum |digit w| for any order. Octal digits from -4 to 3 add up to at most 3.7
        times the number in magnitude (8 - 4 - 4/8 - ..), 4 with the joining of the digits' sums."""
        return (4 * x.shape[-1] * 2.0 ** -23) * (x.abs() @ w.abs().T) + self.rest(x, h) @ w.abs().T

    def change(self, i, codes=None, scales=None):
        """Weights i with codes(nibbles [E, rows, cols]) and scales(codes [E, rows, blocks]) changed."""
        w = self.w[i]
        E, rows, cols = w.codes.shape[0], w.codes.shape[1], w.cols
        c = torch.stack((w.codes & 15, w.codes >> 4), dim=-1).flatten(-2)
        s = ep.untile_fp4_scales(w.scales, E * rows).view(E, rows, -1).clone()
        if codes:
            codes(c)
        if scales:
            scales(s)
        packed = (c[..., 0::2] | c[..., 1::2] << 4).contiguous()
        self.w[i] = ep.FP4(packed, ep.tile_fp4_scales(s), w.format, w.tensor_scale)
        v = F4.values(c.view(-1, cols), s.view(-1, s.shape[-1]), w.format).cuda().view(E, rows, cols)
        if w.tensor_scale is not None:
            v = v * w.tensor_scale.double()[:, None, None]
        self.v[i] = v


def check(layer, x, ids, off):
    """Each element within the bound; off: in the root mean square, relative."""
    scores = torch.rand(ids.shape, device="cuda", generator=gen(3)) + 0.5
    got = layer.run(x, scores, ids, out_dtype=torch.float32)
    want, bound = layer.reference(x, scores, ids, "silu")
    err = (got.double() - want).abs()
    assert err.norm() <= off * want.norm(), float(err.norm() / want.norm())
    assert (err <= bound + 2.0 ** -24 * want.abs()).all()
    assert layer.buf.device_error() == 0
    layer.buf.close()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("blocks", ["all", "one"])
@pytest.mark.parametrize("power", [6, 10, 12])
def test_beside_a_dominant_element_of_x(fmt, blocks, power):
    """One element of 3 x 2^power in every block, or in one of the row, beside unit normals."""
    D, F, E, K, T = 768, 128, 3, 2, 5
    layer = Fine(D, F, E, K, fmt, seed=power)
    n, g = F4.BLOCK[fmt], gen(power)
    at = torch.randint(0, n, (D // n,), device="cuda", generator=g) + torch.arange(0, D, n, device="cuda")
    if blocks == "one":
        at = at[D // n // 2:][:1]

    def zero(c):
        c[..., at] = 0

    layer.change(0, codes=zero)
    x = torch.randn((T, D), device="cuda", generator=g).bfloat16()
    x[:, at] = 3 * 2.0 ** power * (1 - 2 * torch.randint(0, 2, (T, len(at)), device="cuda", generator=g)).bfloat16()
    ids = torch.rand((T, E), device="cuda", generator=g).topk(K, dim=1).indices.to(torch.int32)
    # 3 x 2^12: an element below 1/2 is off by up to 2^-9, 2^-9 / 3^0.5 and of two elements in five in the
    # root mean square: 0.0007 of the projections, at most three times that of the result.
    check(layer, x, ids, 2.0 ** -8)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_beside_a_dominant_element_of_h(fmt):
    """One column of each block of h 2^11 times the others, by its up projection's scales."""
    D, F, E, K, T = 256, 384, 3, 2, 5
    layer = Fine(D, F, E, K, fmt, seed=1)
    n, g = F4.BLOCK[fmt], gen(11)
    at = torch.randint(0, n, (F // n,), device="cuda", generator=g) + torch.arange(0, F, n, device="cuda")

    def large(s):
        s[:, F + at] += 11 if fmt == "mx" else 88

    def zero(c):
        c[..., at] = 0

    layer.change(0, scales=large)
    layer.change(1, codes=zero)
    x = torch.randn((T, D), device="cuda", generator=g).bfloat16()
    ids = torch.rand((T, E), device="cuda", generator=g).topk(K, dim=1).indices.to(torch.int32)
    # h is within 2^-22 of its block's largest, which is at most 2^14 times the others' root mean
    # square (its own magnitude included): 2^-8 / 3^0.5.
    check(layer, x, ids, 2.0 ** -8)


def bf16_layer(gate, up, down):
    """One expert, one column of h for each row of gate and up [128, 2]: x has two elements."""
    buf = ep.Buffer(4, 128, 1, 1, 1)
    w1 = torch.zeros((1, 256, 128), dtype=torch.bfloat16, device="cuda")
    w1[0, :128, :2], w1[0, 128:, :2] = gate, up
    w2 = (torch.eye(128, device="cuda") * down).bfloat16()[None].contiguous()

    def run(x0, x1):
        x = torch.zeros((1, 128), dtype=torch.bfloat16, device="cuda")
        x[0, 0], x[0, 1] = x0, x1
        return buf.moe_layer(x, torch.ones((1, 1), device="cuda"),
                             torch.zeros((1, 1), dtype=torch.int32, device="cuda"), w1, w2,
                             out_dtype=torch.float32)[0]
    return buf, run


def test_h_enters_whole_on_bf16_weights():
    """Gates of 128 or more are silu's own results, so that h is a product of 16 and 8 bits, and a down
    projection of ones gives it back."""
    g = gen(5)
    a, b, c = (torch.randint(lo, 256, (128,), device="cuda", generator=g) for lo in (128, 0, 128))
    gate = torch.stack((a, b), 1).bfloat16()
    up = torch.stack((c, torch.zeros_like(c)), 1).bfloat16()
    buf, run = bf16_layer(gate, up, 1.0)
    want = (a * 256 + b) * c
    assert torch.equal(run(1.0, 2.0 ** -8).double(), want.double() / 256)
    buf.close()


def test_h_above_the_largest_bf16():
    """4095^2 2^104: fp32 holds it, bf16 does not."""
    both = torch.tensor([[255.0, 0.9375]], device="cuda").expand(128, 2).bfloat16()
    buf, run = bf16_layer(both, both, 2.0 ** -10)
    out = run(2.0 ** 56, 2.0 ** 56).double()
    assert torch.equal(out, torch.full_like(out, 4095.0 ** 2 * 2.0 ** 94))
    buf.close()


def test_the_largest_bf16_on_4_bit_weights():
    """x and h of 1.9921875 x 2^127 through weights of 1: every digit's product stays finite."""
    def fp4(rows, at, scale):
        """mx, row r: 1.0 at column at[r], all blocks of the row with this scale code."""
        codes = torch.zeros((rows, 128), dtype=torch.uint8)
        codes[torch.arange(rows), at] = 2
        scales = scale[:, None].expand(rows, 4).to(torch.uint8).contiguous()
        packed = (codes[:, 0::2] | codes[:, 1::2] << 4).contiguous()
        return ep.FP4(packed[None].contiguous().cuda(), ep.tile_fp4_scales(scales.cuda()), "mx")

    # gate: x[0] by 1; up: x[40] = 2^100 by 2^-100, in another block; down: h by 2^-10.
    at = torch.cat((torch.zeros(128, dtype=torch.long), torch.full((128,), 40)))
    w1 = fp4(256, at, torch.cat((torch.full((128,), 127), torch.full((128,), 27))))
    w2 = fp4(128, torch.arange(128), torch.full((128,), 117))
    buf = ep.Buffer(4, 128, 1, 1, 1)
    x = torch.zeros((1, 128), dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[0, 40] = 1.9921875 * 2.0 ** 127, 2.0 ** 100
    out = buf.moe_layer(x, torch.ones((1, 1), device="cuda"),
                        torch.zeros((1, 1), dtype=torch.int32, device="cuda"), w1, w2,
                        out_dtype=torch.float32)[0].double()
    # Columns of h other than a block's own are zeros to w2's rows; each has one.
    assert torch.equal(out, torch.full_like(out, 1.9921875 * 2.0 ** 117))
    assert buf.device_error() == 0
    buf.close()
