"""8-bit AdamW states where one moment of a group leaves fp32's range and the other
does not: the finite one keeps its definition, bit for bit (fp64 oracle)."""

import pytest
import torch

from bit_muon_optimizer_b200 import workloads as WL
from oracle import adamw as OA

pytestmark = pytest.mark.gpu

DEV = "cuda"
HP = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, wd=0.1)


def _step(gm, g, old, t):
    """One step of a state (m codes, m scales, v codes, v scales) on the host; the new one."""
    p = torch.zeros(g.numel(), device=DEV)
    st = gm.AdamWState.zeros([p], 8)
    for dst, src in zip((st.m[0], st.mscale[0], st.v[0], st.vscale[0]), old):
        dst.copy_(src)
    st.step.fill_(t - 1)
    gm.AdamWStep(**HP)(st, [p], [g.to(DEV)])
    torch.cuda.synchronize()
    return [x[0].cpu() for x in (st.m, st.mscale, st.v, st.vscale)], st


def _same_codes(got, want):
    live = want % 128 > 0                      # a zero has either sign
    return torch.equal(got[live], want[live]) and bool((got[~live] % 128 == 0).all())


@pytest.mark.parametrize("n", [128 * 96, 128 * 96 + 37])
@pytest.mark.parametrize("every", [1, 128])
def test_v_overflows_and_m_stays(cuda_lib, n, every):
    """Gradients of 1e21 (all of a group, or one of it): (1 - beta2) g^2 passes fp32's
    range, m does not."""
    gm = cuda_lib
    g = WL.random_matrix((n,), 5, std=1e-3)
    g[::every] = WL.random_matrix((n,), 6, std=1.0)[::every].sign() * (2.0 + WL.random_matrix(
        (n,), 7, std=0.3)[::every].abs()) * 1e21
    m0 = WL.random_matrix((n,), 8, std=1e20 if every == 1 else 3e-4).double()
    old = OA.encode8(m0, WL.random_matrix((n,), 9, std=1e-3).double().square())
    old = [x.float() if x.dtype == torch.float64 else x for x in old]
    (cm, sm, _, sv), st = _step(gm, g, old, 4)
    _, m, v = OA.step(torch.zeros(n), g, *OA.decode8(*old), 4, HP["lr"], *HP["betas"], HP["eps"], HP["wd"])
    want = OA.encode8(m, v)
    assert _same_codes(cm, want[0]) and torch.equal(sm, want[1].float())
    assert bool(torch.isposinf(sv).all())
    m1, _ = st.moments()
    assert bool(torch.isfinite(m1[0]).all())


def test_m_is_infinite_and_v_stays(cuda_lib):
    """Groups whose m had become infinite, with ordinary v and gradients: v's codes and
    scales are the definition's, m stays NaN."""
    gm = cuda_lib
    n = 128 * 400
    g = WL.random_matrix((n,), 15, std=1e-3)
    old = OA.encode8(WL.random_matrix((n,), 18, std=3e-4).double(), WL.random_matrix((n,), 19, std=1e-3).double().square())
    old = [x.float() if x.dtype == torch.float64 else x for x in old]
    old[1][:] = float("inf")
    (_, sm, cv, sv), st = _step(gm, g, old, 9)
    _, m, v = OA.step(torch.zeros(n), g, *OA.decode8(*old), 9, HP["lr"], *HP["betas"], HP["eps"], HP["wd"])
    want = OA.encode8(torch.zeros(n), v)
    assert torch.equal(cv, want[2]) and torch.equal(sv, want[3].float())
    assert not bool(torch.isfinite(sm).any()) and not bool(torch.isfinite(st.moments()[0][0]).any())
