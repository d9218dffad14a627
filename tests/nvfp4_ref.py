"""Caches held in 4 bits, plainly: rows quantised and read in 64 bits, where
every quotient's border and every value is exact."""
from __future__ import annotations

import torch

MAGNITUDES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def e4m3_values():
    """All 256 codes from their fields: bias 7, subnormals, NaN at 0x7f and 0xff."""
    code = torch.arange(256)
    e, m = (code >> 3) & 15, (code & 7).double()
    v = torch.where(e > 0, 2.0 ** (e.double() - 7) * (1 + m / 8), m * 2.0 ** -9)
    v[(code & 0x7f) == 0x7f] = float("nan")
    return torch.where(code >= 128, -v, v)


E4M3 = e4m3_values()


def nearest_even(x, table):
    """Index of the value of an ascending table nearest to x >= 0, ties to the
    even index, past the last one the last."""
    hi = torch.searchsorted(table, x.contiguous()).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - x, x - table[lo]
    take_lo = (down < up) | ((down == up) & (lo % 2 == 0))
    return torch.where(take_lo & (x < table[hi]), lo, hi)


def quantise(x, g):
    """Rows [.., dim] (16-bit types): code bytes [.., dim / 2], scale bytes
    [.., dim / 16]."""
    x = x.double().unflatten(-1, (-1, 16))
    amax = x.abs().amax(-1)
    fine = torch.isfinite(x).all(-1)
    scale = nearest_even(torch.where(fine, amax / (6 * g), 0.0), E4M3[:0x7f])
    d = torch.where(fine, E4M3[scale] * g, 0.0)[..., None]
    # (compared with the table's multiples of d, which are exact)
    size = torch.where(d > 0, torch.where(fine[..., None], x, 0.0).abs() / d.clamp(min=1e-300), 0.0)
    code = nearest_even(size, MAGNITUDES)
    code = torch.where(fine[..., None], code + 8 * ((x < 0) & (d > 0)), 0).flatten(-2)
    scale = torch.where(fine, scale, 0x7f)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), scale.to(torch.uint8)


def values(codes, scales, g):
    """The values of code bytes and scale bytes, in float64."""
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = MAGNITUDES[code & 7] * (1 - 2 * (code >> 3)).double()
    return (v.unflatten(-1, (-1, 16)) * E4M3[scales.long()][..., None]).flatten(-2) * g
