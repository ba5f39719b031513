"""Microscaled 4-bit operands without a GPU: the oracle by hand-worked blocks and by
its bounds, sizes, and every refusal (all before any launch)."""

import ctypes
import math

import pytest
import torch

from bit_muon_optimizer_b200 import gmuon as gm
from oracle import mx4 as OM


def test_oracle_hand_worked_mx_block():
    x = torch.zeros(1, 1, 32)
    x[0, 0, :8] = torch.tensor([5.0, -5.1, 2.5, 3.5, 0.25, -0.26, 7.9, 1.25])   # max 7.9: scale 1
    codes, byte, gs = OM.quant(x, "mx")
    assert gs is None and int(byte[0, 0, 0]) == 127 and byte.shape == (1, 1, 4)
    # ties: 5 -> 4, 2.5 -> 2, 3.5 -> 4, .25 -> 0, 1.25 -> 1; 7.9 saturates
    assert OM.values(codes, byte, gs, 8, "mx")[0, 0].tolist() == [4, -6, 2, 4, 0, -.5, 6, 1]
    x[0, 0, 6] = 8.0                                                            # scale 2
    codes, byte, _ = OM.quant(x, "mx")
    assert int(byte[0, 0, 0]) == 128 and float(OM.values(codes, byte, None, 8, "mx")[0, 0, 6]) == 8
    assert int(OM.quant(torch.full((1, 1, 1), 1e-45), "mx")[1][0, 0, 0]) == 0
    assert int(OM.quant(torch.full((1, 1, 1), math.inf), "mx")[1][0, 0, 0]) == 255


def test_oracle_hand_worked_nv_block():
    x = torch.zeros(1, 2, 16)
    x[0, 0, 0], x[0, 1, 0], x[0, 1, 1] = 2688.0, 6.0, 1.0
    codes, byte, gs = OM.quant(x, "nv")
    assert float(gs) == 1.0
    assert int(byte[0, 0, 0]) == 126 and int(byte[0, 1, 0]) == 56               # 448, 1
    assert OM.values(codes, byte, gs, 2, "nv")[0].tolist() == [[2688, 0], [6, 1]]
    z = OM.quant(torch.zeros(1, 1, 16), "nv")
    assert float(z[2]) == 0 and int(z[0].sum()) == 0 and int(z[1].sum()) == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_oracle_round_trip_error(fmt):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(2, 40, 200, generator=g)
    y = OM.round_trip(x, fmt)
    codes, byte, gs = OM.quant(x, fmt)
    top = OM._blocks(x, fmt).abs().amax(-1).repeat_interleave(OM.BLOCK[fmt], -1)[..., :200]
    # mx: 8/6 of the top may saturate to 6/8; nv: top within the e4m3 step of 6 sb
    assert bool(((y - x).abs() <= top * (0.26 if fmt == "mx" else 1 / 6 + 2.0 ** -4)).all())
    again = OM.round_trip(y.float(), fmt) if fmt == "mx" else y
    assert torch.equal(again, y)                                 # what is representable stays
    t = OM.tile_scales(byte)
    assert int(t[1, 0, 0, 7, 1, 2]) == int(byte[1, 39, 2])       # row 39 = 32 + 7


def test_sizes():
    f = gm.lib
    assert f.gm_mx4_codes_bytes(2, 5, 130) == 2 * 5 * 128
    assert f.gm_mx4_scales_bytes(2, 129, 130, gm.GM_MX4) == 2 * 2 * 2 * 512
    assert f.gm_mx4_scales_bytes(2, 129, 130, gm.GM_NV4) == 2 * 2 * 4 * 512
    for B, r, c in [(0, 1, 1), (65536, 1, 1), (1, 0, 1), (1, 1, 0), (1, (1 << 24) + 1, 1), (1, 1 << 24, 1 << 17)]:
        assert f.gm_mx4_codes_bytes(B, r, c) == 0 and f.gm_mx4_scales_bytes(B, r, c, 0) == 0
    assert f.gm_mx4_scales_bytes(1, 1, 1, 2) == 0
    q = gm.Mx4.empty(3, 200, 77, gm.GM_NV4, device="cpu")
    assert q.codes.numel() == f.gm_mx4_codes_bytes(3, 200, 77)
    assert q.scales.numel() == f.gm_mx4_scales_bytes(3, 200, 77, gm.GM_NV4)


def test_c_refusals():
    ok = 4096

    def quant(B=1, m=4, n=40, X=ok, dt=0, rs=40, bs=160, fmt=1, gs=ok, c=ok, s=ok, ct=ok, st=ok):
        return gm.lib.gm_mx4_quant(B, m, n, X, dt, rs, bs, fmt, gs, c, s, ct, st, None)
    for kw in [dict(B=0), dict(m=0), dict(n=0), dict(n=(1 << 24) + 1), dict(X=None), dict(X=4098),
               dict(dt=1, X=4097), dict(dt=3), dict(fmt=2), dict(fmt=-1), dict(rs=39), dict(rs=-1),
               dict(bs=-1), dict(c=None), dict(s=None), dict(ct=None), dict(st=None),
               dict(c=None, s=None, ct=None, st=None), dict(c=4104), dict(s=4104), dict(ct=4104),
               dict(st=4104), dict(gs=None), dict(gs=4098)]:
        assert quant(**kw) == gm.GM_E_ARG, kw

    def deq(B=1, r=4, c=40, fmt=1, codes=ok, sc=ok, gs=ok, out=ok, dt=0):
        return gm.lib.gm_mx4_dequant(B, r, c, fmt, codes, sc, gs, out, dt, None)
    for kw in [dict(B=0), dict(r=0), dict(c=0), dict(fmt=2), dict(dt=5), dict(codes=None), dict(sc=None),
               dict(out=None), dict(codes=4104), dict(sc=4104), dict(out=4104), dict(gs=None)]:
        assert deq(**kw) == gm.GM_E_ARG, kw

    def mm(B=1, M=4, N=5, K=40, fmt=1, a=ok, sa=ok, ga=ok, b=ok, sb=ok, gb=ok, D=ok, dt=0, acc=0):
        return gm.lib.gm_mx4_matmul(B, M, N, K, fmt, a, sa, ga, b, sb, gb, D, dt, acc, None)
    for kw in [dict(B=0), dict(M=0), dict(N=0), dict(K=0), dict(fmt=3), dict(dt=4), dict(acc=2), dict(a=None),
               dict(sa=None), dict(b=None), dict(sb=None), dict(D=None), dict(a=4104), dict(sb=4104),
               dict(D=4104), dict(ga=None), dict(gb=None), dict(gb=4098)]:
        assert mm(**kw) == gm.GM_E_ARG, kw


def test_binding_refusals():
    x = torch.zeros(2, 4, 40)
    q = gm.Mx4.empty(2, 4, 40, gm.GM_NV4, device="cpu")
    r = gm.Mx4.empty(2, 4, 40, gm.GM_MX4, device="cpu")
    cases = [
        (lambda: gm.mx4_quant(x), "CUDA tensor"),
        (lambda: gm.mx4_quant(x.double()), "dtype"),
        (lambda: gm.mx4_quant(x, 2), "fmt"),
        (lambda: gm.mx4_quant(x, rows=False), "one of the two"),
        (lambda: gm.mx4_quant(x[:, :0]), "empty"),
        (lambda: gm.mx4_quant(x[0, 0]), "expected"),
        (lambda: gm.Mx4.empty(1, 2, 3, 7, device="cpu"), "fmt"),
        (lambda: gm.mx4_dequant(q), "CUDA tensor"),
        (lambda: gm.mx4_matmul(q, q), "CUDA tensor"),
        (lambda: gm.Mx4(gm.GM_NV4, 4, 40, q.codes, q.scales).check(), "gscale"),
        (lambda: gm.Mx4(gm.GM_MX4, 4, 40, q.codes, q.scales).check(), "scales: expected shape"),
        (lambda: gm.Mx4(gm.GM_MX4, 4, 140, r.codes, r.scales).check(), "codes: expected shape"),
        (lambda: gm.Mx4(gm.GM_MX4, 4, 40, r.codes[0], r.scales).check(), "codes"),
        (lambda: gm.Mx4(gm.GM_MX4, 4, 40, r.codes.char(), r.scales).check(), "dtype"),
    ]
    for call, msg in cases:
        with pytest.raises(ValueError, match=msg):
            call()
    assert ctypes.sizeof(ctypes.c_size_t) == 8
