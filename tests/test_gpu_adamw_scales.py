"""The scales of 8-bit AdamW states are rounded from the fp64 maximum of their group,
also where several elements share the maximum in fp32: bit for bit, for groups built
from near ties and over many ordinary groups."""

import pytest
import torch

from bit_muon_optimizer_b200 import workloads as WL
from oracle import adamw as OA

pytestmark = pytest.mark.gpu

DEV = "cuda"
HP = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, wd=0.1)
C = 0.37


def _clip(gm):
    return gm.GradNorm(torch.ones(1, device=DEV), torch.full((1,), C, dtype=torch.float64, device=DEV),
                       torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, device=DEV))


def _pairs(of_v, count):
    """Two elements per group, as codes [2, count], bf16 gradients [2, count] and the
    group's scale, whose new m (or v) are equal but for the rounding of that scale to
    fp32; the smaller first."""
    b1, b2 = HP["betas"]
    gen = torch.Generator().manual_seed(11 + of_v)
    levels = OA.root_levels() if of_v else OA.m_levels()
    top = levels.numel() - 1
    ca = torch.randint(top - 20, top + 1, (count,), generator=gen)          # the larger code
    cb = ca - torch.randint(1, 12, (count,), generator=gen)
    ga = (torch.rand(count, generator=gen) * 4e-4 + 1e-4).bfloat16()
    gb = ga + (torch.rand(count, generator=gen) * 1e-3 + 1e-4).bfloat16()   # with the larger gradient
    x, y = ga.double() * C, gb.double() * C
    if of_v:
        scale = ((1 - b2) * (y * y - x * x) / (b2 * (levels[ca] ** 2 - levels[cb] ** 2))).sqrt().float()
        new = lambda c, z: b2 * (levels[c] * scale.double()).square() + (1 - b2) * (z * z)   # noqa: E731
    else:
        scale = ((1 - b1) * (y - x) / (b1 * (levels[ca] - levels[cb]))).float()
        new = lambda c, z: b1 * (levels[c] * scale.double()) + (1 - b1) * z                  # noqa: E731
    da, db = new(ca, x), new(cb, y)
    assert bool(((da - db).abs() <= 2.0 ** -21 * da).all())
    swap = da > db
    codes = torch.where(swap, torch.stack((cb, ca)), torch.stack((ca, cb)))
    grads = torch.where(swap, torch.stack((gb, ga)), torch.stack((ga, gb)))
    return codes, grads, scale


@pytest.mark.parametrize("ragged", [0, 1])
@pytest.mark.parametrize("at", [(0, 1), (1, 0), (3, 90), (90, 3), (7, 127), (64, 63)])
@pytest.mark.parametrize("of_v", [False, True])
@pytest.mark.parametrize("gdt", [torch.bfloat16, torch.float32])
def test_near_ties_of_the_top_element(cuda_lib, of_v, at, ragged, gdt):
    """Two elements at the places `at` of a group, the larger at the second, that fp32
    hardly tells apart (or orders the other way)."""
    gm = cuda_lib
    groups = 600
    codes, grads, scale = _pairs(of_v, groups)
    n = groups * 128
    cm, cv = torch.zeros(n, dtype=torch.uint8), torch.zeros(n, dtype=torch.uint8)
    g = torch.zeros(n, dtype=torch.bfloat16)
    for k in range(2):
        (cv if of_v else cm)[at[k]::128] = codes[k].to(torch.uint8)
        g[at[k]::128] = grads[k]
    other = torch.full((groups,), 1e-4)
    ms, vs = (other, scale) if of_v else (scale, other)
    lead = 1 if ragged else 0                        # gradients off alignment: the other path
    p = torch.zeros(n, device=DEV)
    hold = torch.zeros(n + 1, dtype=gdt, device=DEV)
    gd = hold[lead:lead + n]
    gd.copy_(g)
    st = gm.AdamWState.zeros([p], 8)
    for dst, src in zip((st.m[0], st.mscale[0], st.v[0], st.vscale[0]), (cm, ms, cv, vs)):
        dst.copy_(src)
    gm.AdamWStep(**HP)(st, [p], [gd], clip=_clip(gm))
    torch.cuda.synchronize()
    _, m, v = OA.step(torch.zeros(n), g, *OA.decode8(cm, ms, cv, vs), 1, HP["lr"], *HP["betas"], HP["eps"],
                      HP["wd"], C)
    wm, wsm, wv, wsv = OA.encode8(m, v)
    assert torch.equal(st.mscale[0].cpu(), wsm.float()) and torch.equal(st.vscale[0].cpu(), wsv.float())
    assert torch.equal(st.m[0].cpu() % 128, wm % 128) and torch.equal(st.v[0].cpu(), wv)


@pytest.mark.parametrize("gdt", [torch.bfloat16, torch.float32])
def test_scales_of_many_groups(cuda_lib, gdt):
    """Three steps of 2^19 groups: every scale equals the one of the fp64 formulas,
    computed from the step's own codes, scales and gradients."""
    gm = cuda_lib
    groups = 1 << 19
    n = groups * 128
    gen = torch.Generator(device=DEV).manual_seed(3)
    b1, b2 = HP["betas"]
    p = torch.zeros(n, device=DEV)
    st, step, clip = gm.AdamWState.zeros([p], 8), gm.AdamWStep(**HP), _clip(gm)
    root, mval = OA.root_levels().to(DEV), OA.m_levels().to(DEV)
    for t in range(3):
        g = (torch.randn(n, generator=gen, device=DEV) * 1e-3).to(gdt)
        mc, vc = st.m[0].int(), st.v[0].int()
        m = mval[(mc & 127).clamp_max(126)] * torch.where(mc > 127, -1.0, 1.0).double()
        m = (m.view(-1, 128) * st.mscale[0].double()[:, None]).flatten()
        r = (root[vc].view(-1, 128) * st.vscale[0].double()[:, None]).flatten()
        del mc, vc
        gd = g.double() * C
        m, r = b1 * m + (1 - b1) * gd, b2 * (r * r) + (1 - b2) * (gd * gd)
        sm = (m.abs().view(-1, 128).amax(1) * (1 / 448)).clamp_min(OA.SCALE_FLOOR).float()
        sv = (OA.root(r.view(-1, 128).amax(1).cpu()) * (1 / 1.9375)).clamp_min(OA.SCALE_FLOOR).float().to(DEV)
        del m, r, gd
        step(st, [p], [g], clip=clip)
        torch.cuda.synchronize()
        bad = int((st.mscale[0] != sm).sum()), int((st.vscale[0] != sv).sum())
        assert bad == (0, 0), (t, bad)
