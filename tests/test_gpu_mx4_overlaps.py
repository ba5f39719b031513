"""Operands of the microscaled operators that overlap what is written are refused."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("nv", [False, True])
def test_overlaps_are_refused(cuda_lib, nv):
    gm = cuda_lib
    fmt = gm.GM_NV4 if nv else gm.GM_MX4
    x = torch.randn(1, 256, 256, device=DEV)
    q = gm.mx4_quant(x, fmt)
    codes, scales = q.codes.clone(), q.scales.clone()
    inside = x.view(torch.uint8).flatten()[:codes.numel()].view_as(codes)
    over = gm.Mx4(fmt, 256, 256, inside, torch.empty_like(scales), torch.empty(1, device=DEV) if nv else None)
    room = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    at = gm.Mx4(fmt, 256, 256, room[:codes.numel()].view_as(codes), scales, q.gscale)
    D = room.view(torch.float32)[4096:4096 + 65536].view(1, 256, 256)
    for call in (lambda: gm.mx4_quant(x, fmt, cols=True, out=(q, q)),      # both orientations into one
                 lambda: gm.mx4_quant(x, fmt, out=over),                    # codes over X itself
                 lambda: gm.mx4_matmul(at, q, out=D), lambda: gm.mx4_matmul(q, at, out=D),
                 lambda: gm.mx4_dequant(at, out=D)):
        with pytest.raises(gm.GmuonError, match="overlap"):
            call()
    torch.cuda.synchronize()
    assert torch.equal(q.codes, codes) and torch.equal(q.scales, scales) and int(room.count_nonzero()) == 0
    gm.mx4_matmul(q, q, out=D)            # one operand on both sides is fine
    assert int(D.count_nonzero()) > 0
