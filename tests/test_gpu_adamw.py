"""gm_adamw_step and gm_grad_norm against the fp64 oracle.

Bounds, u = 2^-24 (an fp32 rounding relative to the value): with S = |b1 m| +
|(1 - b1) g| the new m is off by 5 u S (constant, product: 2 u each, c and its
product 2 u, sum u), v by 8 u v, so sqrt(v)/sqrt(bc2) + eps by 8 u, and
p' = p decay - x scale by 2 u |p| + scale (5 u S + 12 u |m|) / denom + u |p'|,
then half a step of p's type. 8-bit codes are those of the unrounded moments:
equal to the oracle's; a scale is off by its top element's error.
"""

import math

import pytest
import torch

from bit_muon_optimizer_b200 import workloads as WL
from oracle import adamw as OA

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
HP = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, wd=0.1)
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _inputs(sizes, pdt, gdt, seed, std=1e-3):
    p = [WL.random_matrix((n,), seed + 2 * i, std=0.02).to(pdt) for i, n in enumerate(sizes)]
    g = [WL.random_matrix((n,), seed + 2 * i + 1, std=std).to(gdt) for i, n in enumerate(sizes)]
    return p, g


def _state(gm, sizes, bits, seed, t0, std=1e-3):
    """A state in mid-training: moments of the gradients' size, t0 steps done."""
    params = [torch.empty(n) for n in sizes]
    st = gm.AdamWState.zeros([x.to(DEV) for x in params], bits)
    st.step.fill_(t0)
    for i, n in enumerate(sizes):
        m = WL.random_matrix((n,), seed + 5000 + i, std=0.3 * std).double()
        v = WL.random_matrix((n,), seed + 9000 + i, std=std).double().square()
        if bits == 32:
            st.m[i].copy_(m)
            st.v[i].copy_(v)
        else:
            for dst, src in zip((st.m[i], st.mscale[i], st.v[i], st.vscale[i]), OA.encode8(m, v)):
                dst.copy_(src)
    return st


def _old(st, i):
    if st.bits == 32:
        return st.m[i].double().cpu(), st.v[i].double().cpu()
    return OA.decode8(*[t[i].cpu() for t in (st.m, st.mscale, st.v, st.vscale)])


def _check_tensor(before, g, p0, p1, st, i, t, c=1.0, copy=None, lr=HP["lr"]):
    m0, v0 = before
    b1, b2 = HP["betas"]
    p, m, v = OA.step(p0.cpu(), g.cpu(), m0, v0, t, lr, b1, b2, HP["eps"], HP["wd"], c)
    S = b1 * m0.abs() + (1 - b1) * g.double().cpu().abs() * c
    bc1, bc2 = 1 - b1 ** t, 1 - b2 ** t
    den = (v / bc2).sqrt() + HP["eps"]
    tol = 3 * U * p0.double().cpu().abs() + lr / bc1 * (5 * U * S + 12 * U * m.abs()) / den
    for got, dt in ((p1, p1.dtype), (copy, None if copy is None else copy.dtype)):
        if got is None:
            continue
        half = 0.0 if dt == F32 else torch.finfo(dt).eps / 2
        tiny = 0.0 if dt == F32 else torch.finfo(dt).smallest_normal * half
        err = (got.double().cpu() - p).abs()
        assert bool((err <= tol * (1 + half) + half * p.abs() + tiny).all()), (i, float((err - tol).max()))
    if st.bits == 32:
        assert bool(((st.m[i].double().cpu() - m).abs() <= 5 * U * S + 2.0 ** -149).all())
        assert bool(((st.v[i].double().cpu() - v).abs() <= 8 * U * v + 2.0 ** -148).all())
        return
    cm, sm, cv, sv = OA.encode8(m, v)
    got = [x[i].cpu() for x in (st.m, st.mscale, st.v, st.vscale)]
    live = cm % 128 > 0                     # a zero has either sign
    assert torch.equal(got[0][live], cm[live]) and bool((got[0][~live] % 128 == 0).all())
    assert torch.equal(got[2], cv)
    grp = lambda x: torch.nn.functional.pad(x, (0, -x.numel() % 128)).view(-1, 128).amax(1)   # noqa: E731
    assert bool(((got[1].double() - sm).abs() <= 5 * U * grp(S) / 448 + 3 * U * sm).all())
    assert bool(((got[3].double() - sv).abs() <= 8 * U * sv).all())


def _run(gm, sizes, pdt, gdt, bits, seed=1, t0=7, steps=2, copy=None, clip=None, std=1e-3, place=None):
    p, g = _inputs(sizes, pdt, gdt, seed, std)
    place = place or (lambda x: x.to(DEV))
    pd = [place(x) for x in p]
    cd = [place(x.to(copy)) for x in p] if copy else None
    st = _state(gm, sizes, bits, seed, t0, std)
    step = gm.AdamWStep(**HP)
    for s in range(steps):
        gd = [place(x) for x in (g if s == 0 else _inputs(sizes, pdt, gdt, seed + 77 * s, std)[1])]
        before = [_old(st, i) for i in range(len(sizes))]
        p0 = [x.clone() for x in pd]
        c, res = 1.0, None
        if clip:
            res = gm.grad_norm(gd, clip)
            n, c = OA.grad_norm([x.cpu() for x in gd], clip)
            assert abs(float(res.norm) - n) <= 2 * U * n
            assert abs(float(res.scale) - c) <= 1e-14 and int(res.status) == 0
        step(st, pd, gd, copies=cd, clip=res)
        torch.cuda.synchronize()
        assert int(st.step) == t0 + s + 1
        for i in range(len(sizes)):
            _check_tensor(before[i], gd[i], p0[i], pd[i], st, i, t0 + s + 1, c, cd[i] if cd else None)
    return st, pd


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt", [(p, g) for p in (F32, BF16, F16) for g in (F32, BF16, F16)])
def test_step_types(cuda_lib, pdt, gdt, bits):
    _run(cuda_lib, [1000, 1, 4096], pdt, gdt, bits)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 127, 128, 129, 255, 1023, 2047, 2048, 2049, 70001])
def test_step_sizes(cuda_lib, n, bits):
    _run(cuda_lib, [n], F32, BF16, bits, copy=BF16)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("clip", [1e-3, 1e6])
def test_step_clipped(cuda_lib, bits, clip):
    _run(cuda_lib, [5000, 33, 768], F32, F32, bits, clip=clip, copy=F16)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_the_zero_state(cuda_lib, bits):
    gm = cuda_lib
    p, g = _inputs([1000, 200], F32, BF16, 3)
    g[0][:500] = 0                      # rows that no token touched: v and m stay zero
    pd, gd = [x.to(DEV) for x in p], [x.to(DEV) for x in g]
    st = gm.AdamWState.zeros(pd, bits)
    for t in (1, 2):
        before = [_old(st, i) for i in range(2)]
        p0 = [x.clone() for x in pd]
        gm.AdamWStep(**HP)(st, pd, gd)
        torch.cuda.synchronize()
        for i in range(2):
            _check_tensor(before[i], gd[i], p0[i], pd[i], st, i, t)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_cross_a_launch(cuda_lib, bits):
    """More tensors than one launch's table holds, lengths 1..~130."""
    _run(cuda_lib, [1 + (37 * i) % 131 for i in range(900)], F32, F32, bits, steps=1)


@pytest.mark.parametrize("bits", [32, 8])
def test_mixed_types_in_one_list(cuda_lib, bits):
    gm = cuda_lib
    sizes = [300, 4097, 128, 1, 999]
    dts = [(F32, BF16), (BF16, BF16), (F32, F32), (F16, F16), (F32, BF16)]
    p = [_inputs([n], a, b, 10 + i)[0][0].to(DEV) for i, (n, (a, b)) in enumerate(zip(sizes, dts))]
    g = [_inputs([n], a, b, 10 + i)[1][0].to(DEV) for i, (n, (a, b)) in enumerate(zip(sizes, dts))]
    st = _state(gm, sizes, bits, 4, 3)
    before, p0 = [_old(st, i) for i in range(5)], [x.clone() for x in p]
    res = gm.grad_norm(g, 0.01)
    n, c = OA.grad_norm([x.cpu() for x in g], 0.01)
    assert abs(float(res.norm) - n) <= 2 * U * n
    gm.AdamWStep(**HP)(st, p, g, clip=res)
    torch.cuda.synchronize()
    assert int(st.step) == 4
    for i in range(5):
        _check_tensor(before[i], g[i], p0[i], p[i], st, i, 4, c)


@pytest.mark.parametrize("bits", [32, 8])
def test_arrays_off_alignment(cuda_lib, bits):
    """Views that start one element into a buffer: the same values, moved singly."""
    def place(x):
        buf = torch.zeros(x.numel() + 9, dtype=x.dtype, device=DEV)
        view = buf[1:1 + x.numel()]
        view.copy_(x)
        return view
    _run(cuda_lib, [700, 129], F32, BF16, bits, copy=BF16, place=place, clip=0.5)


@pytest.mark.parametrize("bits", [32, 8])
def test_neighbours_of_a_tensor_are_left_alone(cuda_lib, bits):
    """Buffers around ragged tensors (parameters, copies, codes, scales) keep their bytes."""
    gm = cuda_lib
    n = 131
    bufs = {k: torch.full((512,), 7, dtype=dt, device=DEV)
            for k, dt in (("p", F32), ("c", BF16), ("m", torch.uint8 if bits == 8 else F32),
                          ("v", torch.uint8 if bits == 8 else F32), ("ms", F32), ("vs", F32))}
    view = {k: b[128:128 + n] for k, b in bufs.items()}
    sc = {k: bufs[k][128:130] for k in ("ms", "vs")}
    st = gm.AdamWState(bits, [view["m"]], [view["v"]], [sc["ms"]] if bits == 8 else [],
                       [sc["vs"]] if bits == 8 else [], torch.zeros(1, dtype=torch.int64, device=DEV))
    gm.AdamWStep(**HP)(st, [view["p"]], [torch.ones(n, device=DEV)], copies=[view["c"]])
    torch.cuda.synchronize()
    for k, b in bufs.items():
        hi = 128 + (2 if k in sc else n)
        assert bool((b[:128] == 7).all()) and bool((b[hi:] == 7).all()), k


@pytest.mark.parametrize("std", [1e-22, 1e-16, 1e-12, 1e8, 1e15])
def test_extreme_gradients_8bit(cuda_lib, std):
    """Where squares near fp32's limits: codes still those of the unrounded moments."""
    _run(cuda_lib, [1500], F32, F32, 8, std=std, steps=1)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dt", [F32, BF16, F16])
def test_nonfinite_gradient_changes_nothing(cuda_lib, bad, dt):
    gm = cuda_lib
    for bits in (32, 8):
        p, g = _inputs([300, 5000], F32, dt, 6)
        g[1][4099] = bad
        pd, gd = [x.to(DEV) for x in p], [x.to(DEV) for x in g]
        st = _state(gm, [300, 5000], bits, 6, 5)
        old, p0 = st.clone(), [x.clone() for x in pd]
        cp = [x.to(BF16) for x in pd]
        res = gm.grad_norm(gd, 1.0)
        gm.AdamWStep(**HP)(st, pd, gd, copies=cp, clip=res)
        torch.cuda.synchronize()
        assert int(res.status) == gm.GM_E_NONFINITE
        assert all(torch.equal(a, b) for a, b in zip(pd, p0))
        assert all(torch.equal(a, b) for a, b in zip(st.tensors(), old.tensors()))
        # the next, finite step works
        gd[1][4099] = 1.0
        gm.AdamWStep(**HP)(st, pd, gd, copies=cp, clip=gm.grad_norm(gd, 1.0, out=res))
        torch.cuda.synchronize()
        assert int(res.status) == 0 and int(st.step) == 6


def test_nonfinite_group_without_the_flag(cuda_lib):
    """Without a flag a NaN enters as the formula has it: its group of 128 becomes NaN
    (8 bits), its element alone (32 bits); the other groups' codes are exact."""
    gm = cuda_lib
    for bad in (math.nan, math.inf):
        p, g = _inputs([1000], F32, F32, 8)
        g[0][130] = bad
        for bits in (32, 8):
            pd = [p[0].to(DEV)]
            st = _state(gm, [1000], bits, 8, 5)
            before = _old(st, 0)
            gm.AdamWStep(**HP)(st, pd, [g[0].to(DEV)])
            m, v = st.moments()
            torch.cuda.synchronize()
            fin = torch.isfinite(m[0]).cpu()
            span = range(128, 256) if bits == 8 else [130]
            assert torch.equal((~fin).nonzero().flatten(), torch.tensor(list(span)))
            keep = torch.ones(1000, dtype=torch.bool)
            keep[128:256] = False
            if bits == 8:
                _, m1, v1 = OA.step(p[0], g[0], *before, 6, HP["lr"], *HP["betas"], HP["eps"], HP["wd"])
                m1[130] = v1[130] = 0
                cm, _, cv, _ = OA.encode8(m1, v1)
                live = keep & (cm % 128 > 0)
                assert torch.equal(st.m[0].cpu()[live], cm[live])
                assert torch.equal(st.v[0].cpu()[keep], cv[keep])


def test_moments_are_what_the_codes_stand_for(cuda_lib):
    gm = cuda_lib
    st = _state(gm, [1, 777, 4096 * 3], 8, 12, 0)
    for i, t in enumerate(st.m):                       # every code, sign and NaN included
        t.copy_((torch.arange(t.numel()) % 256).to(torch.uint8))
        st.v[i].copy_((torch.arange(t.numel()) * 7 % 256).to(torch.uint8))
    m, v = st.moments()
    torch.cuda.synchronize()
    for i in range(3):
        mo, vo = _old(st, i)
        nan = torch.isnan(mo)
        assert torch.equal(torch.isnan(m[i].cpu()), nan)
        assert bool(((m[i].cpu().double() - mo).abs()[~nan] <= U * mo.abs()[~nan]).all())
        assert bool(((v[i].cpu().double() - vo).abs() <= 4 * U * vo).all())


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("sizes", [[1], [7], [16384], [16385, 3], [100003, 1, 5], [3] * 1500])
def test_grad_norm(cuda_lib, dt, sizes):
    gm = cuda_lib
    _, g = _inputs(sizes, F32, dt, 21, std=1.0)
    gd = [x.to(DEV) for x in g]
    n, c = OA.grad_norm(g, 2.0)
    a, b = gm.grad_norm(gd, 2.0), gm.grad_norm(gd, 2.0)
    torch.cuda.synchronize()
    assert abs(float(a.norm) - n) <= 2 * U * n and abs(float(a.scale) - c) <= 1e-14
    assert torch.equal(a.norm, b.norm) and torch.equal(a.scale, b.scale)
    assert float(gm.grad_norm(gd).scale) == 1.0


def test_grad_norm_of_extreme_values(cuda_lib):
    """Squares that fp32 would lose at either end, subnormals, and a norm past fp32."""
    gm = cuda_lib
    for vals, dt in [([1e-30, 3e-30], F32), ([1e-45, 2.8e-45], F32), ([3e38], F32), ([6e-8, 1.2e-7], F16),
                     ([9.2e-41, 1e-38], BF16), ([3e38, 1e38], BF16), ([0.0], F32)]:
        g = torch.tensor(vals, dtype=torch.float64).to(dt)
        n = float(g.double().square().sum().sqrt())
        r = gm.grad_norm([g.to(DEV)])
        assert abs(float(r.norm) - n) <= 2 * U * n + 2.0 ** -150 and int(r.status) == 0
    r = gm.grad_norm([torch.full((4,), 3e38, device=DEV)], 1.0)     # 6e38
    assert int(r.status) == gm.GM_E_NONFINITE and float(r.norm) == math.inf and float(r.scale) == 0.0


def test_learning_rate_from_the_device_under_a_graph(cuda_lib):
    """A captured clip + step, replayed with new gradients and a new rate, equals
    the eager calls bit for bit; another graph on its own state does not disturb it."""
    gm = cuda_lib
    sizes = [1000, 129, 4096]
    for bits in (32, 8):
        p, g = _inputs(sizes, F32, BF16, 31)
        pd, gd = [x.to(DEV) for x in p], [x.to(DEV) for x in g]
        st, lr = _state(gm, sizes, bits, 31, 0), torch.full((1,), 1e-3, device=DEV)
        p2, st2, step = [x.clone() for x in pd], st.clone(), gm.AdamWStep(**HP)
        warm = torch.cuda.Stream()
        with torch.cuda.stream(warm):      # first use of the kernels, on copies
            step(st.clone(), [x.clone() for x in pd], gd, clip=gm.grad_norm(gd, 0.1), lr=lr)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(st, pd, gd, clip=gm.grad_norm(gd, 0.1), lr=lr)
        for s in range(3):
            for x, y in zip(gd, _inputs(sizes, F32, BF16, 40 + s)[1]):
                x.copy_(y)
            lr.fill_(1e-3 / (s + 1))
            graph.replay()
            step(st2, p2, gd, clip=gm.grad_norm(gd, 0.1), lr=float(lr))
        torch.cuda.synchronize()
        assert int(st.step) == int(st2.step) == 3
        assert all(torch.equal(a, b) for a, b in zip(pd + st.tensors(), p2 + st2.tensors()))


def test_side_stream_and_repeatability(cuda_lib):
    gm = cuda_lib
    sizes = [100_000, 77]
    for bits in (32, 8):
        p, g = _inputs(sizes, F32, F32, 51)
        outs = []
        for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
            pd, gd, st = [x.to(DEV) for x in p], [x.to(DEV) for x in g], _state(gm, sizes, bits, 51, 2)
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                gm.AdamWStep(**HP)(st, pd, gd, clip=gm.grad_norm(gd, 1.0))
            torch.cuda.synchronize()
            outs.append(pd + st.tensors())
        assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_refusals_on_the_device(cuda_lib):
    gm = cuda_lib
    p, g = [torch.zeros(64, device=DEV), torch.zeros(8, 8, device=DEV)], [torch.zeros(64, device=DEV)] * 2
    st, step = gm.AdamWState.zeros(p), gm.AdamWStep()
    res = gm.grad_norm(g, 1.0)
    cases = [
        (lambda: step(st, [p[0], p[0]], g), "more than once"),
        (lambda: step(st, p, g[:1]), "expected 2 tensors"),
        (lambda: step(st, p, [g[0], torch.zeros(63, device=DEV)]), "63 elements"),
        (lambda: step(st, p, [g[0], torch.zeros(8, 16, device=DEV)[:, ::2]]), "contiguous"),
        (lambda: step(st, [p[0], p[1].cpu()], g), "CUDA tensor"),
        (lambda: step(gm.AdamWState.zeros(p[:1]), p, g), "m: expected 2"),
        (lambda: step(st, p, g, copies=p[:1]), "copies: expected 2"),
        (lambda: step(st, p, g, clip=res, skip=res.status), "clip brings"),
        (lambda: step(st, p, g, skip=torch.zeros(1, device=DEV)), "skip: expected"),
        (lambda: step(st, p, g, lr=torch.zeros(1)), "lr: expected on"),
        (lambda: gm.grad_norm([torch.zeros(4, device=DEV)] * 1500, out=res), "out.ws"),
    ]
    for call, msg in cases:
        with pytest.raises(ValueError, match=msg):
            call()
    assert int(st.step) == 0


def test_offsets_beyond_32_bits(cuda_lib):
    """One tensor of 2^31 + 300 elements: its last elements and scales equal those of
    a short tensor with the same contents."""
    gm = cuda_lib
    n, tail = (1 << 31) + 300, 300
    p = torch.zeros(n, dtype=BF16, device=DEV)
    g = torch.zeros(n, dtype=BF16, device=DEV)
    ps, gs = _inputs([tail], BF16, BF16, 61)
    p[-tail:].copy_(ps[0])
    g[-tail:].copy_(gs[0])
    st = gm.AdamWState.zeros([p], 8)
    res = gm.grad_norm([g], 0.01)
    gm.AdamWStep(**HP)(st, [p], [g], clip=res)
    pt, gt = [ps[0].to(DEV)], [gs[0].to(DEV)]
    s2 = gm.AdamWState.zeros(pt, 8)
    r2 = gm.grad_norm(gt, 0.01)
    gm.AdamWStep(**HP)(s2, pt, gt, clip=r2)
    torch.cuda.synchronize()
    assert abs(float(res.norm) - float(r2.norm)) <= 2 * U * float(r2.norm)
    assert torch.equal(p[-tail:], pt[0]) and torch.equal(st.m[0][-tail:], s2.m[0])
    assert torch.equal(st.v[0][-tail:], s2.v[0]) and torch.equal(st.mscale[0][-3:], s2.mscale[0])
    assert int(st.m[0][:-tail].count_nonzero()) == 0 and int(p[:-tail].count_nonzero()) == 0


def test_nonfinite_moments_of_a_group(cuda_lib):
    """What a group of 8-bit moments stands for once a NaN or an infinity is in it: m
    NaN; v NaN or infinite (its zeros NaN); step after step, its neighbours as ever."""
    gm = cuda_lib
    for bad, want in ((math.nan, torch.isnan), (math.inf, torch.isposinf), (-math.inf, torch.isposinf)):
        p, g = _inputs([400], F32, F32, 18)
        g[0][200] = bad
        pd, gd, st = [p[0].to(DEV)], [g[0].to(DEV)], _state(gm, [400], 8, 18, 5)
        for _ in range(3):
            gm.AdamWStep(**HP)(st, pd, gd)
            m, v = st.moments()
            torch.cuda.synchronize()
            inside = torch.zeros(400, dtype=torch.bool, device=DEV)
            inside[128:256] = True
            assert torch.equal(torch.isnan(m[0]), inside) and torch.equal(want(v[0]), inside)
            assert bool(torch.isfinite(v[0][~inside]).all())


def test_states_follow_the_definition_for_many_steps(cuda_lib):
    """Ten free-running steps with 8-bit states: codes and scales bit for bit the
    oracle's, which runs in fp64 from its own state (scales kept in fp32)."""
    gm = cuda_lib
    n = 5000
    b1, b2 = HP["betas"]
    p, _ = _inputs([n], F32, BF16, 71)
    pd, st = [p[0].to(DEV)], _state(gm, [n], 8, 71, 20)
    ref = [x[0].cpu() for x in (st.m, st.mscale, st.v, st.vscale)]
    for t in range(21, 31):
        g = _inputs([n], F32, BF16, 100 + t)[1][0]
        gm.AdamWStep(**HP)(st, pd, [g.to(DEV)])
        _, m, v = OA.step(p[0], g, *OA.decode8(*ref), t, HP["lr"], b1, b2, HP["eps"], HP["wd"])
        cm, sm, cv, sv = OA.encode8(m, v)
        ref = [cm, sm.float(), cv, sv.float()]
        torch.cuda.synchronize()
        live = cm % 128 > 0
        assert torch.equal(st.m[0].cpu()[live], cm[live]) and torch.equal(st.v[0].cpu(), cv), t
        assert torch.equal(st.mscale[0].cpu(), ref[1]) and torch.equal(st.vscale[0].cpu(), ref[3]), t


@pytest.mark.parametrize("n", [1, 5, 130])
def test_infinite_scale_of_a_ragged_group(cuda_lib, n):
    """What lies behind a tensor's end stays out of its last group, also when that
    group's scales are infinite: v infinite (not NaN) step after step."""
    gm = cuda_lib
    p, g = _inputs([n], F32, F32, 19)
    g[0][-1] = math.inf
    for t in (F32, BF16):
        pd, gd, st = [p[0].to(DEV)], [g[0].to(t).to(DEV)], _state(gm, [n], 8, 19, 5)
        for _ in range(3):
            gm.AdamWStep(**HP)(st, pd, gd)
            _, v = st.moments()
            torch.cuda.synchronize()
            last = torch.arange(n, device=DEV) // 128 == (n - 1) // 128
            assert torch.equal(torch.isposinf(v[0]), last)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n", [1, 129, 257])
def test_zero_group_of_one_element(cuda_lib, n, dt):
    """A last group of one element that is zero, moments too: its scales are the
    smallest ones, whatever lies behind the gradient's end (here NaN)."""
    gm = cuda_lib
    buf = torch.full((n + 8,), math.nan, dtype=dt, device=DEV)
    g = buf[:n]
    g.copy_(WL.random_matrix((n,), 3, std=1e-3))
    g[n - 1] = 0
    p = torch.ones(n, device=DEV)
    st = gm.AdamWState.zeros([p], 8)
    for _ in range(2):
        gm.AdamWStep(**HP)(st, [p], [g])
    torch.cuda.synchronize()
    assert float(st.mscale[0][-1]) == float(st.vscale[0][-1]) == 2.0 ** -126
    assert int(st.m[0][-1]) == int(st.v[0][-1]) == 0
    assert bool(torch.isfinite(p).all()) and bool(torch.isfinite(st.mscale[0]).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_written_twice_is_refused(cuda_lib, bits):
    gm = cuda_lib
    p, g = [torch.ones(300, device=DEV) for _ in range(2)], [torch.ones(300, device=DEV)] * 2
    step = gm.AdamWStep(**HP)
    names = ["m", "v"] + (["mscale", "vscale"] if bits == 8 else [])
    for name in names:
        st = gm.AdamWState.zeros(p, bits)
        getattr(st, name)[1] = getattr(st, name)[0]
        with pytest.raises(ValueError, match="more than once"):
            step(st, p, g)
    st = gm.AdamWState.zeros(p, bits)
    st.v = st.m
    with pytest.raises(ValueError, match="more than once"):
        step(st, p, g)
    st = gm.AdamWState.zeros(p, bits)
    with pytest.raises(ValueError, match="copies"):
        step(st, p, g, copies=[torch.empty(300, device=DEV, dtype=BF16)] * 2)
    step(st, p, g, copies=p)                      # an fp32 copy may be the parameter itself
    torch.cuda.synchronize()
    assert int(st.step) == 1 and all(bool(torch.isfinite(x).all()) for x in p)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lr", [0.0, -1e-3])
def test_rates_of_zero_and_below(cuda_lib, bits, lr):
    """A rate of zero leaves the parameters bit for bit as they were and moves the
    states; a negative one is the formula's."""
    gm = cuda_lib
    sizes = [1, 129, 5000]
    p, g = _inputs(sizes, F32, F32, 4)
    pd, gd = [x.to(DEV) for x in p], [x.to(DEV) for x in g]
    st = _state(gm, sizes, bits, 4, 7)
    before = [_old(st, i) for i in range(3)]
    gm.AdamWStep(**{**HP, "lr": lr})(st, pd, gd)
    torch.cuda.synchronize()
    for i in range(3):
        if lr == 0.0:
            assert torch.equal(pd[i].cpu(), p[i])
        want, m, v = OA.step(p[i], g[i], *before[i], 8, lr, *HP["betas"], HP["eps"], HP["wd"])
        # as in the module's bounds, with |lr|
        b1, b2 = HP["betas"]
        S = b1 * before[i][0].abs() + (1 - b1) * g[i].double().abs()
        den = (v / (1 - b2 ** 8)).sqrt() + HP["eps"]
        tol = 3 * U * p[i].double().abs() + abs(lr) / (1 - b1 ** 8) * (5 * U * S + 12 * U * m.abs()) / den
        assert bool(((pd[i].double().cpu() - want).abs() <= tol).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_two_streams_step_two_states(cuda_lib, bits):
    """Steps of different states at the same time, one with a norm into a kept
    result, give the bits of steps one after the other."""
    gm = cuda_lib
    sizes = [70001, 129, 1]
    step = gm.AdamWStep(**HP)

    def start(seed):
        p, g = _inputs(sizes, F32, BF16, seed)
        return [x.to(DEV) for x in p], [x.to(DEV) for x in g], _state(gm, sizes, bits, seed, 3)
    ends = []
    for together in (False, True):
        work = [start(s) for s in (11, 12)]
        norms = [gm.grad_norm(g * 40, 1e-3) for _, g, _ in work]       # longer lists than the ones below
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in work]
        for _ in range(3):
            for (p, g, st), s, nrm in zip(work, streams, norms):
                with torch.cuda.stream(s if together else torch.cuda.current_stream()):
                    step(st, p, g, clip=gm.grad_norm(g, 1e-3, out=nrm))
        torch.cuda.synchronize()
        ends.append([t.clone() for p, _, st in work for t in (*p, *st.tensors())])
    for a, b in zip(*ends):
        assert torch.equal(a.view(torch.uint8) if a.dtype == F32 else a, b.view(torch.uint8) if b.dtype == F32 else b)
