"""32-bit AdamW states at either end of fp32's range, and beside the least eps."""

import math

import pytest
import torch
from test_gpu_adamw import DEV, F32, HP, U, _check_tensor, _inputs, _old, _run, _state

from oracle import adamw as OA

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("std", [1e-22, 1e-16, 1e-12, 1e8, 1e15, 1e18])
def test_extreme_gradients(cuda_lib, std):
    _run(cuda_lib, [1500, 1], F32, F32, 32, std=std, steps=1)


@pytest.mark.parametrize("std", [3e19, 1e20])
def test_squares_past_fp32(cuda_lib, std):
    """g^2 is past fp32's range, (1 - beta2) g^2 is not: v is finite and right."""
    gm = cuda_lib
    p, g = _inputs([1500], F32, F32, 2, std=std)
    g[0].clamp_(-5e20, 5e20)
    pd, gd, st = [p[0].to(DEV)], [g[0].to(DEV)], _state(gm, [1500], 32, 2, 4, std=1e18)
    before = [_old(st, 0)]
    gm.AdamWStep(**HP)(st, pd, gd)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(st.v[0]).all())
    _check_tensor(before[0], gd[0], p[0], pd[0], st, 0, 5)


@pytest.mark.parametrize("std", [1e-24, 1e-23, 1e-22, 1e-21, 1e-20])
def test_the_least_eps_beside_what_fp32_loses_of_v(cuda_lib, std):
    """A v below fp32's numbers is zero. Its root, q = sqrt(2^-149 / bc2) at most, then
    moves an update m / (r + eps) by no more than its share q / eps."""
    gm = cuda_lib
    eps = 1e-18
    p, g = _inputs([3000], F32, F32, 4, std=std)
    p[0].zero_()
    pd, gd = [p[0].to(DEV)], [g[0].to(DEV)]
    st = gm.AdamWState.zeros(pd)
    b1, b2 = HP["betas"]
    gm.AdamWStep(**{**HP, "eps": eps})(st, pd, gd)
    torch.cuda.synchronize()
    z = torch.zeros(3000)
    want, m, v = OA.step(z, g[0], z, z, 1, HP["lr"], b1, b2, eps, HP["wd"])
    bc1, bc2 = 1 - b1, 1 - b2
    den = (v / bc2).sqrt() + eps
    q = math.sqrt(2.0 ** -149 / bc2)
    # roundings as in the ordinary bounds, g and m near fp32's subnormals (2^-149), v's loss
    rel = 5 * U + 12 * U + q / eps
    tol = HP["lr"] / bc1 * (rel * m.abs() + 2.0 ** -148) / (den - q).clamp_min(eps)
    assert bool(((pd[0].double().cpu() - want).abs() <= tol).all())
