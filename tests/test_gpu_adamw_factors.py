"""Gradient factors near and past either end of fp32's range: what a clip of a huge norm
gives. The step is the formula's with the factor in fp64 (bounds and oracle as in the
ordinary tests of the step)."""

import pytest
import torch
from test_gpu_adamw import DEV, F16, F32, HP, _check_tensor, _inputs, _old, _state

from oracle import adamw as OA

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [1.0, 1e-3, 1e-12])
def test_clip_of_a_huge_norm(cuda_lib, bits, max_norm):
    """fp32 gradients around 1e36: the clip factor is below fp32's normal numbers."""
    gm = cuda_lib
    sizes = [70000, 33, 4096]
    p, g = _inputs(sizes, F32, F32, 3, std=1e36)
    pd, gd = [x.to(DEV) for x in p], [x.to(DEV) for x in g]
    st = _state(gm, sizes, bits, 3, 6, std=1e-2 * max_norm)
    before = [_old(st, i) for i in range(3)]
    res = gm.grad_norm(gd, max_norm)
    gm.AdamWStep(**HP)(st, pd, gd, clip=res)
    torch.cuda.synchronize()
    c = float(res.scale)
    want = OA.grad_norm(g, max_norm)[1]
    assert abs(c - want) <= 1e-12 * want and c < 2.0 ** -120
    for i in range(3):
        _check_tensor(before[i], gd[i], p[i], pd[i], st, i, 7, c)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("c,std", [(1.2e-38, 1e36), (1e-60, 1e36), (1e-300, 1.0), (0.0, 1.0), (1e30, 1e-33),
                                   (3e38, 1e-40), (1e45, 1e-43), (2.0 ** 120, 1e-37)])
def test_any_factor(cuda_lib, bits, c, std):
    gm = cuda_lib
    sizes = [5000, 130]
    p, g = _inputs(sizes, F32, F32, 13, std=std)
    pd, gd = [x.to(DEV) for x in p], [x.to(DEV) for x in g]
    cp = [x.to(F16) for x in pd]
    st = _state(gm, sizes, bits, 13, 6, std=1e-2)
    before = [_old(st, i) for i in range(2)]
    clip = gm.GradNorm(torch.ones(1, device=DEV), torch.full((1,), c, dtype=torch.float64, device=DEV),
                       torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, device=DEV))
    gm.AdamWStep(**HP)(st, pd, gd, clip=clip, copies=cp)
    torch.cuda.synchronize()
    for i in range(2):
        _check_tensor(before[i], gd[i], p[i], pd[i], st, i, 7, c, cp[i])
