"""AdamW with moments in 32 or 8 bits, in plain fp64 on the CPU.

Decoupled weight decay (Loshchilov and Hutter, "Decoupled Weight Decay
Regularization"), bias-corrected moments (Kingma and Ba, "Adam"). The 8-bit
formats are the library's own, read from their definition: the value of every
code is listed, and a number takes the nearest listed value (ties to the even
code).
"""

import math

import numpy as np
import torch

GROUP = 128
SCALE_FLOOR = 2.0 ** -126


def m_levels():
    """Values of the codes 0..126 of e4m3 (3 fraction bits, exponents from -6)."""
    return torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10)
                         for c in range(127)], dtype=torch.float64)


def root_levels():
    """Values of the codes 0..255 that keep sqrt(v) (4 fraction bits, exponents -14..0)."""
    return torch.tensor([(c & 15) * 2.0 ** -18 if c < 16 else (16 + (c & 15)) * 2.0 ** ((c >> 4) - 19)
                         for c in range(256)], dtype=torch.float64)


def nearest(a, levels):
    """Index of the level nearest to each a >= 0 (levels ascending; ties to the even index)."""
    hi = torch.searchsorted(levels, a).clamp(1, levels.numel() - 1)
    lo = hi - 1
    dl, dh = a - levels[lo], levels[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.where(up, hi, lo)


def root(v):
    """The correctly rounded fp64 root (torch's on the CPU may be off in the last
    place, which moves a quotient off a true tie)."""
    return torch.from_numpy(np.sqrt(v.numpy()))


def _groups(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % GROUP)).view(-1, GROUP)


def encode8(m, v):
    """(m codes uint8, m scales, v codes uint8, v scales) of flat fp64 moments."""
    n = m.numel()
    mg, vg = _groups(m.double()), _groups(v.double())
    rg = root(vg)
    # products with the reciprocals, as the definition has it: at a true tie of a
    # code's quotient the last place of the scale decides
    sm = (mg.abs().amax(1) * (1 / 448)).clamp_min(SCALE_FLOOR)
    sv = (rg.amax(1) * (1 / 1.9375)).clamp_min(SCALE_FLOOR)
    cm = nearest((mg / sm[:, None]).abs(), m_levels()) + 128 * (mg < 0).long()
    cv = nearest(rg / sv[:, None], root_levels())
    cv = torch.maximum(cv, (vg.float() > 0).long())
    flat = lambda c: c.flatten()[:n].to(torch.uint8)                        # noqa: E731
    return flat(cm), sm, flat(cv), sv


def decode8(cm, sm, cv, sv):
    """fp64 (m, v) of codes and scales."""
    at = torch.arange(cm.numel()) // GROUP
    cm, cv = cm.long(), cv.long()
    m = m_levels()[(cm & 127).clamp_max(126)] * torch.where(cm > 127, -1.0, 1.0) * sm.double()[at]
    m[(cm & 127) == 127] = math.nan
    r = root_levels()[cv] * sv.double()[at]
    return m, r * r


def grad_norm(grads, max_norm=math.inf):
    """(norm, clip factor) of a list of gradients."""
    n = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    return n, min(1.0, max_norm / (n + 1e-6))


def step(p, g, m, v, t, lr, beta1, beta2, eps, wd, c=1.0):
    """The t-th step (t = 1 first) of one tensor: new (p, m, v), all fp64."""
    g = g.double() * c
    m = beta1 * m.double() + (1 - beta1) * g
    v = beta2 * v.double() + (1 - beta2) * (g * g)
    mh, vh = m / (1 - beta1 ** t), v / (1 - beta2 ** t)
    return p.double() - lr * (mh / (vh.sqrt() + eps) + wd * p.double()), m, v
