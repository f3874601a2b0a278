"""Microscaled 4-bit floating point in 64 bits on the CPU, for the tests: written from the format's
definition, apart from the kernels."""
import math

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
BLOCK = {"mx": 32, "nv": 16}
NAN_CODE = {"mx": 255, "nv": 127}


def e4m3_table() -> torch.Tensor:
    """The values of the codes 0..126."""
    c = torch.arange(127)
    e, m = c >> 3, (c & 7).double()
    return torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))


def nearest_even(v: torch.Tensor, table: torch.Tensor) -> torch.Tensor:
    """Index of the entry of an ascending table nearest to each v >= 0, the even one of two."""
    hi = torch.searchsorted(table, v).clamp(1, len(table) - 1)
    lo = hi - 1
    down, up = v - table[lo], table[hi] - v
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantize(x: torch.Tensor, fmt: str, g: float = 1.0):
    """(codes 0..15 [rows, cols], scale codes [rows, blocks]) of x [rows, cols] on the CPU."""
    v = x.double().cpu().unflatten(-1, (-1, BLOCK[fmt]))
    most = v.abs().amax(-1)
    bad = ~torch.isfinite(most)
    most = torch.where(bad, 0.0, most)
    v = torch.where(bad[..., None], 0.0, v)
    if fmt == "mx":
        e = torch.frexp(most).exponent - 1
        code = (e - 2 + 127).clamp(0, 254)
        code = torch.where(most > 0, code, 0)
        unit = torch.exp2(code.double() - 127)
    else:
        code = nearest_even((most / (6 * g)).clamp(max=448), e4m3_table())
        unit = e4m3_table()[code] * g
    a = torch.where(unit[..., None] > 0, v.abs() / unit[..., None], 0.0)
    q = nearest_even(a.clamp(max=6), GRID)
    # The sign of what rounds to zero is not part of the value.
    q = torch.where((v < 0) & (q > 0), q + 8, q)
    code = torch.where(bad, NAN_CODE[fmt], code)
    return q.flatten(-2).to(torch.uint8), code.to(torch.uint8)


def values(q: torch.Tensor, code: torch.Tensor, fmt: str, g: float = 1.0) -> torch.Tensor:
    """What codes 0..15 [rows, cols] and scale codes [rows, blocks] stand for, in 64 bits."""
    q, code = q.cpu().long(), code.cpu().long()
    s = torch.exp2(code.double() - 127) if fmt == "mx" else e4m3_table()[code.clamp(max=126)]
    s = torch.where(code == NAN_CODE[fmt], torch.nan, s) * g
    v = torch.where(q >= 8, -GRID[q % 8], GRID[q % 8])
    return (v.unflatten(-1, (-1, BLOCK[fmt])) * s[..., None]).flatten(-2)


def unpack(codes: torch.Tensor) -> torch.Tensor:
    """Codes 0..15 [rows, cols] from bytes [rows, cols / 2]; -0 as 0."""
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).cpu()
    return torch.where(c == 8, 0, c)


def random_fp4(gen: torch.Generator, lead: tuple, cols: int, fmt: str, scale: float = 1.0):
    """(packed codes, row-major scale codes) on the GPU: every element, scales of a few binades."""
    codes = torch.randint(0, 256, (*lead, cols // 2), dtype=torch.uint8, device="cuda", generator=gen)
    r = torch.randint(0, 3, (*lead, cols // BLOCK[fmt]), device="cuda", generator=gen)
    e = round(math.log2(scale))
    if fmt == "mx":
        return codes, (127 + e - r).to(torch.uint8)
    m = torch.randint(0, 8, r.shape, device="cuda", generator=gen)
    return codes, ((max(3, 7 + e) - r) * 8 + m).to(torch.uint8)
