"""Lists of mixed types: refused as a whole, before the step is counted or any tensor
moved; stepped, they are what the lists of each type give."""

import pytest
import torch

from bit_muon_optimizer_b200 import workloads as WL

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def test_a_refused_list_changes_nothing(cuda_lib):
    """65537 tensors of one combination of types behind one of another."""
    gm = cuda_lib
    n = 65537
    flat = [torch.full((n,), 0.5, device=DEV) for _ in range(3)]
    head = torch.ones(130, device=DEV, dtype=BF16)
    p = [head, *flat[0].split(1)]
    g = [torch.ones(130, device=DEV), *torch.ones(n, device=DEV).split(1)]
    st = gm.AdamWState(32, [torch.ones(130, device=DEV), *flat[1].split(1)],
                       [torch.ones(130, device=DEV), *flat[2].split(1)], [], [],
                       torch.full((1,), 3, dtype=torch.int64, device=DEV))
    with pytest.raises(gm.GmuonError, match="65537"):
        gm.AdamWStep(lr=0.1)(st, p, g)
    torch.cuda.synchronize()
    assert int(st.step) == 3
    assert bool((head == 1).all()) and bool((st.m[0] == 1).all()) and all(bool((f == 0.5).all()) for f in flat)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("copies", [False, True])
def test_all_combinations_in_one_list(cuda_lib, bits, copies):
    """Two tensors of each of the 27 combinations (9 without copies), shuffled: bit for
    bit the steps of the lists of one combination."""
    gm = cuda_lib
    types = [(a, b, c) for a in (F32, BF16, F16) for b in (F32, BF16, F16) for c in ((F32, BF16, F16) if copies else (None,))]
    types = types[::2] + types[1::2] + types[::-1]
    step = gm.AdamWStep(lr=1e-2)
    p = [WL.random_matrix((100 + 67 * i,), i, std=0.02).to(a).to(DEV) for i, (a, _, _) in enumerate(types)]
    g = [WL.random_matrix((100 + 67 * i,), 900 + i, std=1e-3).to(b).to(DEV) for i, (_, b, _) in enumerate(types)]
    c = [torch.zeros(x.numel(), dtype=t[2], device=DEV) for x, t in zip(p, types)] if copies else None
    st = gm.AdamWState.zeros(p, bits)
    p1 = [x.clone() for x in p]
    c1 = [x.clone() for x in c] if copies else None
    alone = [gm.AdamWState.zeros([x], bits) for x in p1]
    clip = gm.grad_norm(g, 0.5)
    for _ in range(2):
        step(st, p, g, copies=c, clip=clip)
        for i, s in enumerate(alone):
            step(s, p1[i:i + 1], g[i:i + 1], copies=c1[i:i + 1] if copies else None, clip=clip)
    torch.cuda.synchronize()
    assert int(st.step) == 2
    for i, s in enumerate(alone):
        assert torch.equal(p[i], p1[i]) and (not copies or torch.equal(c[i], c1[i])), types[i]
        assert all(torch.equal(a[i], b[0]) for a, b in ((st.m, s.m), (st.v, s.v)))
        assert bits == 32 or torch.equal(st.mscale[i], s.mscale[0]) and torch.equal(st.vscale[i], s.vscale[0])
