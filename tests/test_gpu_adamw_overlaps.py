"""Lists whose arrays overlap are refused before anything is changed."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gdt", [(F32, F32), (F32, BF16)])
def test_overlapping_arrays_are_refused(cuda_lib, bits, gdt):
    gm = cuda_lib
    flat = torch.ones(900, device=DEV)
    p = [flat[:300], flat[300:600]]
    g = [torch.ones(300, dtype=t, device=DEV) for t in gdt]
    st, step = gm.AdamWState.zeros(p, bits), gm.AdamWStep(lr=0.1)
    big = torch.zeros(400, device=DEV)
    calls = [
        lambda: step(st, p, g, copies=[p[1], p[0]]),
        lambda: step(st, p, g, copies=[flat[600:], flat[599:899]]),
        lambda: step(st, [flat[:300], flat[299:599]], g),
        lambda: step(st, p, [flat[1:301], g[1]]),
        lambda: step(st, p, g, copies=[g[0], big[:300]]) if gdt[0] == F32 else step(st, p, [p[1], p[0]]),
    ]
    if bits == 32:
        calls.append(lambda: step(st, p, g, copies=[st.m[1], st.v[0]]))
    for call in calls:
        with pytest.raises(gm.GmuonError, match="overlap"):
            call()
    torch.cuda.synchronize()
    assert int(st.step) == 0 and bool((flat == 1).all())
    # what stays allowed: neighbours, a copy that is its own parameter, one gradient for both
    step(st, p, [g[0], g[0]], copies=p)
    torch.cuda.synchronize()
    assert int(st.step) == 1 and torch.equal(p[0], p[1]) and bool((flat[600:] == 1).all())


def test_overlapping_moments_are_refused(cuda_lib):
    gm = cuda_lib
    st = gm.AdamWState.zeros([torch.zeros(300, device=DEV)], 8)
    o = torch.zeros(700, device=DEV)
    for m, v in ((o[:300], o[:300]), (o[:300], o[299:599]), (o[:300], st.mscale[0][:1].expand(300))):
        with pytest.raises((gm.GmuonError, ValueError), match="overlap|contiguous"):
            st.moments(out=([m], [v]))
    m, v = st.moments(out=([o[:300]], [o[300:600]]))
    torch.cuda.synchronize()
    assert bool((o == 0).all())
