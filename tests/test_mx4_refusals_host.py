"""Microscaled operands that overlap what is written beside them, by the C entry points
(every call is refused)."""

import pytest
import torch

from bit_muon_optimizer_b200 import gmuon as gm

MB = 1 << 20
B, R, C = 2, 128, 256          # codes 2 x 128 x 128 = 32 KB, scales 2 or 4 KB, X 256 KB in fp32


def _refused(status):
    assert status == gm.GM_E_ARG and b"overlap" in gm.lib.gm_last_error(), gm.lib.gm_last_error()


@pytest.mark.parametrize("fmt", [0, 1])
def test_quantisation(fmt):
    at = dict(X=MB, gs=2 * MB, c=3 * MB, s=4 * MB, ct=5 * MB, st=6 * MB)

    def call(**kw):
        a = {**at, **kw}
        return gm.lib.gm_mx4_quant(B, R, C, a["X"], 0, C, R * C, fmt, a["gs"], a["c"], a["s"], a["ct"], a["st"], None)
    for kw in [dict(ct=3 * MB), dict(st=4 * MB), dict(c=4 * MB), dict(c=MB), dict(c=MB + 4 * B * R * C - 16),
               dict(st=MB + 16), dict(s=3 * MB + 128 * R * B - 16), dict(ct=6 * MB - 16)]:
        _refused(call(**kw))
    if fmt:
        for kw in [dict(gs=3 * MB), dict(gs=MB + 4), dict(gs=6 * MB + 64)]:
            _refused(call(**kw))


@pytest.mark.parametrize("fmt", [0, 1])
def test_decoding(fmt):
    n = 4 * B * R * C
    for out in [3 * MB, 3 * MB + 64, 3 * MB - n + 16, 4 * MB] + [2 * MB - n + 16] * fmt:
        _refused(gm.lib.gm_mx4_dequant(B, R, C, fmt, 3 * MB, 4 * MB, 2 * MB, out, 0, None))


@pytest.mark.parametrize("fmt", [0, 1])
def test_product(fmt):
    n = 4 * B * R * R                 # D of 128 x 128
    for out in [2 * MB, 2 * MB - n + 16, 3 * MB + 16, 4 * MB, 5 * MB] + [6 * MB - 16, 7 * MB - 16] * fmt:
        _refused(gm.lib.gm_mx4_matmul(B, R, R, C, fmt, 2 * MB, 3 * MB, 6 * MB, 4 * MB, 5 * MB, 7 * MB, out, 0, 0, None))


def _meets(lo, hi, B, m, n, rs, bs):
    """Whether the bytes lo .. hi meet rows of n bytes, by listing the rows."""
    return any(lo < b * bs + r * rs + n and hi > b * bs + r * rs for b in range(B) for r in range(m))


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls that are in order would run on these addresses")
@pytest.mark.parametrize("B,m,n,rs,bs", [(1, 5, 16, 24, 0), (3, 4, 16, 16, 96), (2, 3, 16, 40, 200), (3, 1, 32, 32, 64),
                                         (2, 4, 16, 24, 0), (3, 2, 16, 64, 16)])
def test_outputs_in_the_gaps_of_a_strided_matrix(B, m, n, rs, bs):
    """gscale (4 B bytes) at every place around the rows (fp32, sizes here in bytes): refused
    as overlapping exactly where it meets a row; else the call gets as far as the device."""
    base, seen = 1 << 20, set()
    for off in range(-16, (B - 1) * bs + m * rs + 16, 4):
        status = gm.lib.gm_mx4_quant(B, m, n // 4, base, 0, rs // 4, bs // 4, 1, base + off, 3 * base, 4 * base, None,
                                     None, None)
        meets = _meets(off, off + 4 * B, B, m, n, rs, bs)
        seen.add(meets)
        assert status in ((gm.GM_E_ARG,) if meets else (gm.GM_E_CUDA, gm.GM_E_UNSUPPORTED)), off   # no device here
    assert seen == {True, False}
