"""Microscaled 4-bit floating point in plain fp64 on the CPU.

Elements e2m1 and power-of-two scales of 32-element blocks as in the OCP
Microscaling Formats specification (MXFP4, its conversion with scale exponent
floor(log2 max) - 2); the two-level form has 16-element blocks with an e4m3 scale
under one fp32 scale of the matrix. Every rounding is the nearest of a listed set
(ties to the even code); divisions here cannot cross a border: a border times the
scales has at most 31 bits, so a quotient that is not on it is 2^-31 away, and fp64
keeps 2^-53.
"""

import math

import torch

from .adamw import m_levels, nearest

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
BLOCK = {"mx": 32, "nv": 16}


def _blocks(x, fmt):
    """[B, m, Kp / block, block] fp64, zeros behind the last column."""
    x = torch.nn.functional.pad(x.double(), (0, -x.shape[-1] % 128))
    return x.unflatten(-1, (-1, BLOCK[fmt]))


def quant(x, fmt):
    """codes [B, m, Kp] (0..15), scale bytes [B, m, Kp / block], gscale [B] or None of
    x [B, m, n]."""
    xb = _blocks(x, fmt)
    top = xb.abs().amax(-1)
    if fmt == "mx":
        bad = ~torch.isfinite(top)
        _, e = torch.frexp(torch.where(bad, 1.0, top))
        byte = torch.where(top > 0, (e.long() - 1 + 125).clamp_min(0), 0)
        scale = torch.ldexp(torch.ones_like(top), byte - 127)
        byte = torch.where(bad, 255, byte)
        z = torch.where(bad[..., None], 0.0, xb / scale[..., None])
        gs = None
    else:
        gs = (xb.abs().amax((-1, -2, -3)) / 2688).float()
        gs = torch.where(torch.isfinite(gs), gs, math.nan)
        g = gs.double()[:, None, None]
        t = torch.where(g > 0, top / (6 * g), 0.0)
        byte = nearest(t.clamp_max(448.0), m_levels())
        s = m_levels()[byte] * g
        z = torch.where((s > 0)[..., None], xb / s[..., None], 0.0)
    code = nearest(z.abs().clamp_max(6.0), E2M1)
    return (code + 8 * ((z < 0) & (code > 0)).long()).flatten(-2), byte, gs


def values(codes, byte, gs, cols, fmt):
    """The fp64 numbers that codes and scales stand for, [B, m, cols]."""
    mag = E2M1[codes & 7] * torch.where(codes > 7, -1.0, 1.0).double()
    if fmt == "mx":
        s = torch.ldexp(torch.ones(byte.shape, dtype=torch.float64), byte - 127)
        s = torch.where(byte == 255, math.nan, s)
    else:
        s = m_levels()[byte] * gs.double()[:, None, None]
    return (mag.unflatten(-1, (-1, BLOCK[fmt])) * s[..., None]).flatten(-2)[..., :cols]


def round_trip(x, fmt):
    """What x becomes, [B, m, n]."""
    return values(*quant(x, fmt), x.shape[-1], fmt)


def tile_scales(byte):
    """Scale bytes [B, rows, nb] in the operand's layout, by its formula, entry by entry."""
    B, rows, nb = byte.shape
    out = torch.zeros((B, -(-rows // 128), nb // 4, 32, 4, 4), dtype=torch.uint8)
    for r in range(rows):
        for j in range(nb):
            out[:, r // 128, j // 4, r % 32, r % 128 // 32, j % 4] = byte[:, r, j].to(torch.uint8)
    return out


def pack(codes):
    """Packed codes [B, rows, Kp / 2]."""
    return (codes[..., 0::2] + 16 * codes[..., 1::2]).to(torch.uint8)
