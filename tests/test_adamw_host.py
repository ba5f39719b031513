"""The AdamW step and the gradient norm without a GPU: the oracle against torch's
own AdamW and against its definition, and every refusal of the binding and of the
C entry points (all before any launch)."""

import ctypes
import math

import numpy as np
import pytest
import torch

from bit_muon_optimizer_b200 import gmuon as gm
from oracle import adamw as OA


def test_oracle_step_is_torch_adamw():
    g = torch.Generator().manual_seed(0)
    p = torch.randn(300, generator=g, dtype=torch.float64)
    ref = torch.nn.Parameter(p.clone())
    opt = torch.optim.AdamW([ref], lr=3e-3, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.2)
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    for t in range(1, 6):
        grad = torch.randn(300, generator=g, dtype=torch.float64)
        ref.grad = grad.clone()
        opt.step()
        p, m, v = OA.step(p, grad, m, v, t, 3e-3, 0.8, 0.95, 1e-6, 0.2)
        assert torch.allclose(p, ref.detach(), rtol=1e-12, atol=1e-14)


def test_oracle_levels_and_rounding():
    ml, rl = OA.m_levels(), OA.root_levels()
    e4m3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(ml, e4m3) and ml[-1] == 448
    assert rl[255] == 1.9375 and rl[16] == 2.0 ** -14 and rl[1] == 2.0 ** -18
    assert bool((rl[1:] > rl[:-1]).all())
    for levels in (ml, rl):
        assert torch.equal(OA.nearest(levels, levels), torch.arange(levels.numel()))
        mid = (levels[1:] + levels[:-1]) / 2          # ties: the even index of each pair
        i = torch.arange(mid.numel())
        assert torch.equal(OA.nearest(mid, levels), i + i % 2)


def test_oracle_codec_round_trip_bounds():
    g = torch.Generator().manual_seed(1)
    m = torch.randn(1000, generator=g, dtype=torch.float64) * 1e-4
    v = torch.randn(1000, generator=g, dtype=torch.float64).square() * 1e-7
    v[::7] = 0
    m2, v2 = OA.decode8(*OA.encode8(m, v))
    at = torch.arange(1000) // 128
    _, sm, _, sv = OA.encode8(m, v)
    # half a step: 2^-4 of the value, or of the smallest normal below it
    assert bool(((m2 - m).abs() <= torch.maximum(m.abs() * 2.0 ** -4, sm[at] * 2.0 ** -10)).all())
    r, r2 = v.sqrt(), v2.sqrt()
    assert bool(((r2 - r).abs() <= torch.maximum(r * 2.0 ** -5, sv[at] * 2.0 ** -18)).all())
    assert torch.equal(v2 == 0, v == 0)               # what is not zero does not become zero


def _call(fn, *args):
    return fn(*args), gm.lib.gm_last_error()


def test_c_refusals():
    ok = 4096
    prm = lambda **kw: gm.AdamWParams(**{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.0,   # noqa: E731
                                                bits=32, clip=None, lr_dev=None), **kw})
    row = lambda **kw: np.array([[kw.get("p", ok), kw.get("g", ok), kw.get("m", ok), kw.get("v", ok),   # noqa: E731
                                  kw.get("ms", 0), kw.get("vs", 0), kw.get("copy", 0),
                                  kw.get("numel", 8)]], dtype=np.int64)

    def step(count=1, table=row(), pdt=0, gdt=0, cdt=0, p=prm(), st=ok, skip=None, scratch=ok):
        return gm.lib.gm_adamw_step(count, None if table is None else table.ctypes.data, pdt, gdt, cdt,
                                    ctypes.byref(p), st, skip, scratch, None)
    bad = [
        dict(count=0), dict(count=65537), dict(table=None), dict(pdt=3), dict(gdt=-1), dict(cdt=9),
        dict(table=row(numel=0)), dict(table=row(numel=-5)), dict(table=row(p=0)), dict(table=row(g=0)),
        dict(table=row(m=0)), dict(table=row(v=0)), dict(table=row(p=4098)), dict(table=row(g=4097)),
        dict(table=row(m=4098)), dict(pdt=1, table=row(p=4097)), dict(cdt=1, table=row(copy=4097)),
        dict(p=prm(bits=16)), dict(p=prm(bits=8)),                          # no scales
        dict(p=prm(bits=8), table=row(ms=ok, vs=4098)),
        dict(p=prm(lr=math.nan)), dict(p=prm(wd=math.inf)), dict(p=prm(beta1=1.0)),
        dict(p=prm(beta2=-0.1)), dict(p=prm(beta1=math.nan)), dict(p=prm(eps=0.0)),
        dict(p=prm(eps=math.inf)), dict(p=prm(clip=4100)), dict(p=prm(lr_dev=4098)),
        dict(st=None), dict(st=4100), dict(skip=4098), dict(scratch=None), dict(scratch=4104),
    ]
    for kw in bad:
        assert step(**kw) == gm.GM_E_ARG, kw
    # the largest count's workspace, and none outside the range
    assert gm.lib.gm_grad_norm_workspace_bytes(0) == 0
    assert gm.lib.gm_grad_norm_workspace_bytes(65537) == 0
    need = gm.lib.gm_grad_norm_workspace_bytes(1)
    assert 0 < need < gm.lib.gm_grad_norm_workspace_bytes(65536)
    grad = lambda g=ok, n=8, dt=0: np.array([[g, n, dt]], dtype=np.int64)    # noqa: E731

    def norm(count=1, table=grad(), mx=1.0, out=ok, scale=ok, status=ok, ws=ok, nb=need):
        return gm.lib.gm_grad_norm(count, None if table is None else table.ctypes.data, mx, out, scale,
                                   status, ws, nb, None)
    for kw in [dict(count=0), dict(count=65537), dict(table=None), dict(mx=0.0), dict(mx=-1.0),
               dict(mx=math.nan), dict(out=None), dict(scale=None), dict(status=None),
               dict(table=grad(g=0)), dict(table=grad(n=0)), dict(table=grad(dt=3)),
               dict(table=grad(g=4098)), dict(table=grad(g=4097, dt=1))]:
        assert norm(**kw) == gm.GM_E_ARG, kw
    for kw in [dict(ws=None), dict(nb=need - 1), dict(ws=4096 + 128)]:
        assert norm(**kw) == gm.GM_E_WORKSPACE, kw
    un = lambda t, c=1: gm.lib.gm_adamw_unpack8(c, t.ctypes.data, None)      # noqa: E731
    full = np.full((1, 7), ok, dtype=np.int64)
    for col in range(6):
        t = full.copy()
        t[0, col] = 0
        assert un(t) == gm.GM_E_ARG
    t = full.copy()
    t[0, 6] = 0
    assert un(t) == gm.GM_E_ARG and un(full, 0) == gm.GM_E_ARG
    t = full.copy()
    t[0, 4] = 4098
    assert un(t) == gm.GM_E_ARG


def test_binding_refusals():
    p = [torch.zeros(5), torch.zeros(3, 4)]
    g = [torch.zeros(5), torch.zeros(3, 4)]
    st = gm.AdamWState.zeros(p)
    step = gm.AdamWStep()
    cases = [
        (lambda: step(st, [], []), "non-empty"),
        (lambda: step(st, p[0], g), "list of tensors"),
        (lambda: step(st, [x.double() for x in p], g), r"params\[0\]: dtype"),
        (lambda: step(st, [torch.zeros(0)], [torch.zeros(0)]), "0 elements"),
        (lambda: step(st, p, g), "expected a CUDA tensor"),
        (lambda: gm.grad_norm([]), "non-empty"),
        (lambda: gm.grad_norm(torch.zeros(4)), "list of tensors"),
        (lambda: gm.grad_norm([torch.zeros(4, dtype=torch.int32)]), "dtype"),
        (lambda: gm.grad_norm([torch.zeros(4), torch.zeros(0)]), "expected a CUDA tensor|0 elements"),
        (lambda: gm.AdamWState(16, [], [], [], [], torch.zeros(1)), "32 or 8"),
        (lambda: gm.AdamWState.zeros([]), "non-empty"),
        (lambda: gm.AdamWState.zeros(p, 4), "32 or 8"),
        (lambda: st.moments(out=([], [])), "own tensors"),
    ]
    for call, msg in cases:
        with pytest.raises(ValueError, match=msg):
            call()


def test_zero_states_have_their_layout():
    p = [torch.zeros(1), torch.zeros(129), torch.zeros(300, 7)]
    a, b = gm.AdamWState.zeros(p), gm.AdamWState.zeros(p, 8)
    assert [t.numel() for t in a.m] == [1, 129, 2100] and a.mscale == []
    assert all(t.dtype == torch.uint8 for t in b.m + b.v)
    assert [t.numel() for t in b.vscale] == [1, 2, 17]
    for st in (a, b):
        assert all(t.data_ptr() % 16 == 0 for t in st.tensors())
        assert all(bool((t == 0).all()) for t in st.tensors())
        c = st.clone()
        assert c.bits == st.bits and c.m[0].data_ptr() != st.m[0].data_ptr()


@pytest.mark.parametrize("bits,least", [(32, 1e-30), (8, 1e-12)])
def test_least_eps(bits, least):
    """An eps beside which the 8-bit step's root, zero for a v below 2^-126, would
    matter is refused."""
    table = np.array([[4096] * 6 + [0, 8]], dtype=np.int64)
    for eps in (least * 0.99, 0.0, -1.0, math.nan):
        prm = gm.AdamWParams(1e-3, 0.9, 0.999, eps, 0.0, bits, None, None)
        assert gm.lib.gm_adamw_step(1, table.ctypes.data, 0, 0, 0, ctypes.byref(prm), 4096, None, 4096,
                                    None) == gm.GM_E_ARG
        assert b"eps" in gm.lib.gm_last_error()
