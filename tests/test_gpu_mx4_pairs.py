"""The two operands of a GM_NV4 matrix share its scale: neither is rewritten alone."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_one_of_a_pair_is_not_rewritten_alone(cuda_lib):
    gm = cuda_lib
    x, x2 = torch.randn(2, 96, 70, device=DEV), torch.randn(2, 96, 70, device=DEV) * 50
    q, qt = gm.mx4_quant(x, gm.GM_NV4, cols=True)
    before = gm.mx4_dequant(q), gm.mx4_dequant(qt)
    with pytest.raises(ValueError, match="pair"):
        gm.mx4_quant(x2, gm.GM_NV4, out=q)
    with pytest.raises(ValueError, match="pair"):
        gm.mx4_quant(x2, gm.GM_NV4, rows=False, cols=True, out=qt)
    assert torch.equal(gm.mx4_dequant(q), before[0]) and torch.equal(gm.mx4_dequant(qt), before[1])
    # together, and into operands of their own
    gm.mx4_quant(x2, gm.GM_NV4, cols=True, out=(q, qt))
    alone = gm.Mx4.empty(2, 96, 70, gm.GM_NV4, torch.device(DEV))
    gm.mx4_quant(x2, gm.GM_NV4, out=alone)
    gm.mx4_quant(x2, gm.GM_NV4, out=alone)
    assert torch.equal(gm.mx4_dequant(q), gm.mx4_dequant(alone))
    single = gm.mx4_quant(x, gm.GM_NV4)
    gm.mx4_quant(x2, gm.GM_NV4, out=single)
    assert torch.equal(gm.mx4_dequant(single), gm.mx4_dequant(alone))


def test_pairs_made_by_hand(cuda_lib):
    gm = cuda_lib
    x = torch.randn(1, 40, 130, device=DEV)
    q = gm.Mx4.empty(1, 40, 130, gm.GM_NV4, torch.device(DEV))
    qt = gm.Mx4.empty(1, 130, 40, gm.GM_NV4, torch.device(DEV), gscale=q.gscale)
    with pytest.raises(ValueError, match="pair"):
        gm.mx4_quant(x, gm.GM_NV4, rows=False, cols=True, out=qt)
    gm.mx4_quant(x, gm.GM_NV4, cols=True, out=(q, qt))
    for kw in (dict(out=q), dict(out=qt, rows=False, cols=True)):
        with pytest.raises(ValueError, match="pair"):
            gm.mx4_quant(x, gm.GM_NV4, **kw)


def test_gm_mx4_pairs_share_nothing(cuda_lib):
    gm = cuda_lib
    x, x2 = torch.randn(1, 64, 64, device=DEV), torch.randn(1, 64, 64, device=DEV)
    q, qt = gm.mx4_quant(x, cols=True)
    before = gm.mx4_dequant(qt)
    gm.mx4_quant(x2, out=q)
    assert torch.equal(gm.mx4_dequant(qt), before) and torch.equal(gm.mx4_dequant(q), gm.mx4_dequant(gm.mx4_quant(x2)))
