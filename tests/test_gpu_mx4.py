"""Microscaled 4-bit operands against the fp64 oracle.

Codes and scales are defined by exact quotients, so they are compared bit for bit.
A product's sum is fp32: K / 64 steps of the tensor cores (or fewer in parallel,
joined), each of which drops at most 2^-22 of the sum of magnitudes S = |A| |B|^T it
adds to; then half a step of D's type, plus, for GM_NV4, three roundings of the
matrix scales. Where every product and sum is a multiple of 1/4 below 2^22 nothing is
dropped and D is exact.
"""

import math

import pytest
import torch

from bit_muon_optimizer_b200 import workloads as WL
from oracle import mx4 as OM

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
FMTS = ["mx", "nv"]


def _fmt(gm, fmt):
    return gm.GM_MX4 if fmt == "mx" else gm.GM_NV4


def _random(shape, seed, dtype=F32, std=1.0):
    """Gaussian entries, a few columns 20 times as large."""
    x = WL.random_matrix(shape, seed, std=std)
    x[..., ::37] *= 20
    return x.to(dtype)


def _check(gm, q, x, fmt):
    """Operand q holds exactly what the oracle makes of x [B, m, n] (on the host)."""
    codes, byte, gs = OM.quant(x, fmt)
    B, m, n = x.shape
    assert (q.rows, q.cols) == (m, n)
    got = q.codes.cpu()
    lo, hi = (got & 15).long(), (got >> 4).long()
    mine = torch.stack((lo, hi), -1).flatten(-2)
    mine = torch.where(mine == 8, 0, mine)                    # a zero has either sign
    assert torch.equal(mine, codes)
    assert torch.equal(q.scales.cpu(), OM.tile_scales(byte))
    if fmt == "nv":
        assert torch.equal(q.gscale.cpu().view(torch.int32)[~torch.isnan(gs)], gs.view(torch.int32)[~torch.isnan(gs)])
        assert torch.equal(torch.isnan(q.gscale.cpu()), torch.isnan(gs))
    v = OM.values(codes, byte, gs, n, fmt)
    nan = torch.isnan(v)
    for dt in (F32, BF16, F16):
        y = gm.mx4_dequant(q, dtype=dt).cpu()
        assert torch.equal(torch.isnan(y), nan)
        tol = (U * (1 if fmt == "nv" else 0) + (0 if dt == F32 else torch.finfo(dt).eps / 2 + U)) * v.abs()
        tiny = 2.0 ** -149 if dt == F32 else torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
        top = torch.finfo(dt).max
        ok = (y.double() - v).abs() <= tol + (tiny if dt != F32 or fmt == "nv" else 0)
        ok |= (v.abs() > top) & torch.isinf(y)
        assert bool(ok[~nan].all()), (dt, float((y.double() - v).abs()[~nan].max()))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 1, 2050), (2, 3, 7), (1, 128, 128), (1, 129, 130), (3, 33, 257),
                                   (1, 200, 1023), (1, 1, 128), (2, 300, 64), (1, 17, 31)])
def test_quant_is_exact(cuda_lib, fmt, dtype, shape):
    gm = cuda_lib
    x = _random(shape, 5 + shape[-1], dtype)
    xd = x.to(DEV)
    f = _fmt(gm, fmt)
    xt = x.transpose(-1, -2).contiguous()
    q = gm.mx4_quant(xd, f)
    both = gm.mx4_quant(xd, f, cols=True)
    qt = gm.mx4_quant(xd, f, rows=False, cols=True)
    torch.cuda.synchronize()
    for mine, host in ((q, x), (both[0], x), (both[1], xt), (qt, xt)):
        _check(gm, mine, host.float(), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale", [1e-44, 1e-38, 3e-37, 1e-30, 1e-20, 1e20, 1e30, 1.5e37])
def test_quant_over_fp32s_range(cuda_lib, fmt, scale):
    gm = cuda_lib
    x = (_random((1, 40, 96), 3, std=1.0).clamp(-20, 20).double() * scale).float()
    x[0, 7] = 0
    _check(gm, gm.mx4_quant(x.to(DEV), _fmt(gm, fmt)), x, fmt)
    _check(gm, gm.mx4_quant(x.to(DEV), _fmt(gm, fmt), rows=False, cols=True), x.transpose(-1, -2), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_quant_at_the_borders(cuda_lib, fmt):
    """Values on, just below and just above every rounding border, both signs; block
    maxima on the borders of the e4m3 scale."""
    gm = cuda_lib
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    near = torch.cat([mids, torch.nextafter(mids, mids * 0), torch.nextafter(mids, mids * 9)])
    row = torch.zeros(1, 8, 128)
    vals = torch.cat([near, -near])                    # 42 values
    for r, s in enumerate([1.0, 2.0 ** -9, 0.75, 448.0, 0.8125, 3.0, 1 / 3, 1e-3]):
        for b in range(8):
            part = vals[b * 6:(b + 1) * 6]
            row[0, r, b * 16:b * 16 + len(part)] = part * s
            row[0, r, b * 16 + 15] = 6.0 * s
    row[0, 3, 127] = 2688.0                            # nv: gscale 1, scales exact or rounded
    _check(gm, gm.mx4_quant(row.to(DEV), _fmt(gm, fmt)), row, fmt)
    # block maxima 6 * (borders of e4m3 and their neighbours): the scale's own rounding
    levels = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (levels[1:] + levels[:-1]) / 2 * 6
    tops = torch.cat([mid, torch.nextafter(mid, mid * 0), torch.nextafter(mid, mid * 9)])
    x = torch.zeros(1, 48, 128)
    x.view(-1, 16)[:len(tops), 3] = tops
    x[0, 47, 127] = 2688.0
    _check(gm, gm.mx4_quant(x.to(DEV), _fmt(gm, fmt)), x, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_nonfinite_values(cuda_lib, fmt, bad):
    gm = cuda_lib
    x = _random((2, 40, 100), 8)
    x[1, 5, 50] = bad
    for q, h in zip(gm.mx4_quant(x.to(DEV), _fmt(gm, fmt), cols=True), (x, x.transpose(-1, -2))):
        _check(gm, q, h, fmt)
        nan = torch.isnan(gm.mx4_dequant(q).cpu())
        assert not bool(nan[0].any())
        assert int(nan[1].sum()) == (4000 if fmt == "nv" else 32 if q.cols == 100 else 32)


@pytest.mark.parametrize("fmt", FMTS)
def test_strided_inputs(cuda_lib, fmt):
    """Slices of a wider buffer (rows on and off 16 bytes), an expanded batch."""
    gm = cuda_lib
    wide = _random((2, 50, 400), 9, BF16).to(DEV)
    for a, b in [(0, 130), (8, 200), (3, 77), (133, 400)]:
        v = wide[:, 1:, a:b]
        _check(gm, gm.mx4_quant(v, _fmt(gm, fmt)), v.cpu().float(), fmt)
        _check(gm, gm.mx4_quant(v, _fmt(gm, fmt), rows=False, cols=True), v.cpu().float().transpose(-1, -2), fmt)
    e = wide[:1].expand(3, -1, -1)
    _check(gm, gm.mx4_quant(e, _fmt(gm, fmt)), e.cpu().float(), fmt)
    for bad in (wide.transpose(1, 2), wide[..., ::2], wide[:, :1].expand(-1, 4, -1)):
        with pytest.raises(ValueError, match="adjacent"):
            gm.mx4_quant(bad, _fmt(gm, fmt))


@pytest.mark.parametrize("fmt", FMTS)
def test_quant_into_buffers_and_graph(cuda_lib, fmt):
    gm = cuda_lib
    f = _fmt(gm, fmt)
    x = _random((1, 70, 90), 10).to(DEV)
    out = gm.mx4_quant(x, f, cols=True)
    x2 = _random((1, 70, 90), 11).to(DEV)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        gm.mx4_quant(x, f, cols=True, out=out)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        gm.mx4_quant(x, f, cols=True, out=out)
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    _check(gm, out[0], x2.cpu(), fmt)
    _check(gm, out[1], x2.cpu().transpose(-1, -2), fmt)
    with pytest.raises(ValueError, match="out"):
        gm.mx4_quant(x[:, :69], f, out=out[0])
    if fmt == "nv":
        other = gm.mx4_quant(x, f, rows=False, cols=True)
        with pytest.raises(ValueError, match="share one gscale"):
            gm.mx4_quant(x, f, cols=True, out=(out[0], other))


def _values(gm, q):
    """fp64 of an operand from its own codes, by the oracle's tables."""
    c = q.codes.cpu().long()
    codes = torch.stack((c & 15, c >> 4), -1).flatten(-2)
    nb = q.scales.shape[2] * 4
    byte = q.scales.cpu().permute(0, 1, 4, 3, 2, 5).reshape(c.shape[0], -1, nb)[:, :q.rows].long()
    fmt = "mx" if q.fmt == gm.GM_MX4 else "nv"
    return OM.values(codes, byte, q.gscale.cpu() if fmt == "nv" else None, q.cols, fmt)


def _check_product(gm, A, Bm, got, before=None):
    a, b = _values(gm, A).to(DEV), _values(gm, Bm).to(DEV)
    want = a @ b.transpose(-1, -2)
    S = a.abs() @ b.abs().transpose(-1, -2)
    if before is not None:
        want, S = want + before.double(), S + before.double().abs()
    dt = got.dtype
    half = U if dt == F32 else torch.finfo(dt).eps / 2
    tol = (math.ceil(A.cols / 64) + 2) * 2.0 ** -22 * S + half * want.abs()
    tiny = 0.0 if dt == F32 else torch.finfo(dt).smallest_normal * half
    err = (got.double() - want).abs()
    assert bool((err <= tol + tiny).all()), (float((err / (S + 1e-300)).max()), A.rows, Bm.rows, A.cols)


SIZES = [(1, 1, 1), (1, 16, 32), (5, 3, 7), (16, 256, 512), (128, 256, 256), (129, 257, 130), (128, 128, 64),
         (300, 200, 1000), (1, 3584, 2048), (7, 500, 4100), (1000, 773, 771), (64, 64, 16384), (257, 1025, 33),
         # enough tiles for CTA pairs: one tile a pair, several, ragged ends, short and odd K
         (2048, 1500, 200), (1700, 2053, 771), (4096, 5632, 2048), (5000, 3000, 100), (129, 9500, 640)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(cuda_lib, fmt, M, N, K):
    gm = cuda_lib
    f = _fmt(gm, fmt)
    A = gm.mx4_quant(_random((1, M, K), 1, BF16).to(DEV), f)
    Bm = gm.mx4_quant(_random((1, N, K), 2, F32, std=0.05).to(DEV), f)
    for dt in (F32, BF16, F16):
        D = gm.mx4_matmul(A, Bm, out_dtype=dt)
        assert D.shape == (1, M, N) and D.dtype == dt
        _check_product(gm, A, Bm, D)
    again = gm.mx4_matmul(A, Bm, out_dtype=F16)
    assert torch.equal(D, again)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(3, 5, 7), (128, 256, 256), (130, 300, 1030), (1, 600, 9000), (400, 900, 512),
                                   (2500, 1300, 1030), (3000, 6000, 256)])
def test_product_of_small_multiples_is_exact(cuda_lib, fmt, M, N, K):
    """Entries that are e2m1 numbers, scales all one: every sum is a multiple of 1/4
    below 2^22, so fp32 holds each step and D equals the fp64 product bit for bit."""
    gm = cuda_lib
    f = _fmt(gm, fmt)
    g = torch.Generator().manual_seed(K)
    mk = lambda r: OM.E2M1[torch.randint(0, 8, (1, r, K), generator=g)] * \
        (1 - 2 * torch.randint(0, 2, (1, r, K), generator=g))                # noqa: E731
    ops = []
    for r in (M, N):
        v = mk(r)
        codes = (torch.searchsorted(OM.E2M1, v.abs()) + 8 * (v < 0).long())
        codes = torch.nn.functional.pad(codes, (0, -K % 128))
        q = gm.Mx4.empty(1, r, K, f, DEV)
        q.codes.copy_(OM.pack(codes))
        q.scales.fill_(127 if fmt == "mx" else 56)
        if fmt == "nv":
            q.gscale.fill_(1.0)
        ops.append((q, v))
    D = gm.mx4_matmul(ops[0][0], ops[1][0], out_dtype=F32)
    assert torch.equal(D.cpu().double(), ops[0][1] @ ops[1][1].transpose(-1, -2))


@pytest.mark.parametrize("M,pad", [(260, 0), (2600, 1500)])
@pytest.mark.parametrize("fmt", FMTS)
def test_product_places_every_scale(cuda_lib, fmt, M, pad):
    """One non-zero element per row with its own block scale: D shows each scale byte."""
    gm = cuda_lib
    f = _fmt(gm, fmt)
    K = 1024
    blk = OM.BLOCK[fmt]
    nb = K // blk
    N = nb + pad                                                # more columns: CTA pairs
    g = torch.Generator().manual_seed(7)
    A, Bm = gm.Mx4.empty(1, M, K, f, DEV), gm.Mx4.empty(1, N, K, f, DEV)
    codes = torch.zeros(1, M, K, dtype=torch.long)
    codes[..., ::blk] = 2                                       # 1.0 at the head of every block
    byte = torch.randint(100, 150, (1, M, nb), generator=g) if fmt == "mx" else \
        torch.randint(1, 127, (1, M, nb), generator=g)
    A.codes.copy_(OM.pack(codes))
    A.scales.copy_(OM.tile_scales(byte))
    sel = torch.zeros(1, N, K, dtype=torch.long)
    sel[0, torch.arange(N), torch.arange(N) % nb * blk] = 2     # row j picks block j mod nb
    Bm.codes.copy_(OM.pack(sel))
    sb = torch.randint(100, 150, (1, N, nb), generator=g) if fmt == "mx" else \
        torch.randint(1, 127, (1, N, nb), generator=g)
    Bm.scales.copy_(OM.tile_scales(sb))
    if fmt == "nv":
        A.gscale.fill_(1.0)
        Bm.gscale.fill_(1.0)
    D = gm.mx4_matmul(A, Bm, out_dtype=F32)
    assert torch.equal(D.cpu().double(), _values(gm, A) @ _values(gm, Bm).transpose(-1, -2))


@pytest.mark.parametrize("fmt", FMTS)
def test_product_batched_accumulated(cuda_lib, fmt):
    gm = cuda_lib
    f = _fmt(gm, fmt)
    for B, M, N, K in [(3, 40, 70, 200), (2, 130, 260, 300), (5, 1, 256, 4096), (3, 1000, 1031, 300),
                       (2, 1100, 1536, 700)]:
        A = gm.mx4_quant(_random((B, M, K), 1).to(DEV), f)
        Bm = gm.mx4_quant(_random((B, N, K), 2, std=0.1).to(DEV), f)
        for dt in (F32, BF16, F16):
            D0 = _random((B, M, N), 3, dt).to(DEV)
            D = D0.clone()
            gm.mx4_matmul(A, Bm, out=D, accumulate=True)
            _check_product(gm, A, Bm, D, D0)


@pytest.mark.parametrize("fmt", FMTS)
def test_product_leaves_its_neighbours_alone(cuda_lib, fmt):
    gm = cuda_lib
    f = _fmt(gm, fmt)
    M, N, K = 131, 77, 200
    A, Bm = gm.mx4_quant(_random((1, M, K), 1).to(DEV), f), gm.mx4_quant(_random((1, N, K), 2).to(DEV), f)
    for dt in (F32, F16):
        buf = torch.full((M * N + 512,), 7.0, dtype=dt, device=DEV)
        D = buf[256:256 + M * N].view(1, M, N)
        gm.mx4_matmul(A, Bm, out=D)
        _check_product(gm, A, Bm, D)
        assert bool((buf[:256] == 7).all()) and bool((buf[256 + M * N:] == 7).all())


@pytest.mark.parametrize("fmt", FMTS)
def test_product_of_nonfinite_operands(cuda_lib, fmt):
    """A NaN in X makes its row of D NaN (mx) or its matrix (nv), no other."""
    gm = cuda_lib
    f = _fmt(gm, fmt)
    x = _random((2, 140, 300), 1)
    x[1, 9, 33] = math.nan
    D = gm.mx4_matmul(gm.mx4_quant(x.to(DEV), f), gm.mx4_quant(_random((2, 90, 300), 2).to(DEV), f),
                      out_dtype=F32).cpu()
    nan = torch.isnan(D)
    want = torch.zeros_like(nan)
    want[1, 9 if fmt == "mx" else slice(None)] = True
    assert torch.equal(nan, want)
    # behind the last row and column: garbage scales there reach nothing
    A, Bm = gm.mx4_quant(x[:1].to(DEV), f), gm.mx4_quant(_random((1, 90, 300), 2).to(DEV), f)
    ref = gm.mx4_matmul(A, Bm, out_dtype=F32)
    for q in (A, Bm):
        s = q.scales.view(1, -1, q.scales.shape[2], 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
        flat = torch.arange(s.shape[1] * 128, device=DEV).view(s.shape[1], 4, 32)
        s[:, flat >= q.rows] = 255 if fmt == "mx" else 127
    assert torch.equal(gm.mx4_matmul(A, Bm, out_dtype=F32), ref)


@pytest.mark.parametrize("fmt", FMTS)
def test_products_on_two_streams_and_in_a_graph(cuda_lib, fmt):
    gm = cuda_lib
    f = _fmt(gm, fmt)
    ops = [(gm.mx4_quant(_random((1, 4, 16384), s).to(DEV), f),
            gm.mx4_quant(_random((1, 700, 16384), s + 50).to(DEV), f)) for s in range(4)]
    ref = [gm.mx4_matmul(*o, out_dtype=F32) for o in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(r) for r in ref]
    for rep in range(3):
        for i, o in enumerate(ops):
            with torch.cuda.stream(streams[i % 2]):
                gm.mx4_matmul(*o, out=outs[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gm.mx4_matmul(*ops[i], out=outs[i])
        graphs.append(g)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for i, g in enumerate(graphs * 2):          # two graphs at a time
        with torch.cuda.stream(streams[i % 2]):
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(outs[i], ref[i]) for i in range(2))


def test_product_refusals_on_the_device(cuda_lib):
    gm = cuda_lib
    x = _random((1, 20, 256), 1).to(DEV)
    A, V = gm.mx4_quant(x), gm.mx4_quant(x, gm.GM_NV4)
    cases = [
        (lambda: gm.mx4_matmul(A, V), "differ"),
        (lambda: gm.mx4_matmul(A, gm.mx4_quant(x[..., :255])), "differ"),
        (lambda: gm.mx4_matmul(A, gm.mx4_quant(x.expand(2, -1, -1))), "differ"),
        (lambda: gm.mx4_matmul(A, A, accumulate=True), "needs out"),
        (lambda: gm.mx4_matmul(A, A, out=torch.empty(1, 20, 19, device=DEV)), "out: expected shape"),
        (lambda: gm.mx4_matmul(A, A, out=torch.empty(1, 20, 20, device=DEV, dtype=torch.int32)), "dtype"),
        (lambda: gm.mx4_matmul(A, A, out=torch.empty(1, 20, 40, device=DEV)[..., ::2]), "contiguous"),
        (lambda: gm.mx4_dequant(A, out=torch.empty(1, 20, 255, device=DEV)), "out: expected shape"),
    ]
    for call, msg in cases:
        with pytest.raises(ValueError, match=msg):
            call()


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_layers_step_ends_in_the_optimizers(cuda_lib, fmt):
    """The operators as they are used together: a linear layer's forward and backward
    products in 4 bits, the weight gradient clipped by the global norm and taken by
    a GRASP step (the weight) and by AdamW (a vector), the new weight quantised."""
    gm = cuda_lib
    f = _fmt(gm, fmt)
    T, m, n, k = 300, 128, 256, 8
    X, dY = _random((1, T, n), 1, BF16).to(DEV), _random((1, T, m), 2, BF16, std=1e-2).to(DEV)
    W = _random((1, m, n), 3, std=0.02).to(DEV)
    bias, gbias = torch.zeros(m, device=DEV), dY.float().sum((0, 1))
    Xq, XT = gm.mx4_quant(X, f, cols=True)
    Wq, WT = gm.mx4_quant(W, f, cols=True)
    Yq, YT = gm.mx4_quant(dY, f, cols=True)
    for got, a, b in ((gm.mx4_matmul(Xq, Wq), Xq, Wq), (gm.mx4_matmul(Yq, WT), Yq, WT),
                      (gm.mx4_matmul(YT, XT, out_dtype=F32), YT, XT)):
        _check_product(gm, a, b, got)
    G = gm.mx4_matmul(YT, XT, out_dtype=F32)
    res = gm.grad_norm([G, gbias], 1.0)
    n2 = math.sqrt(float(G.double().square().sum() + gbias.double().square().sum()))
    assert abs(float(res.norm) - n2) <= 2 * U * n2
    step, st = gm.GraspStep(1, m, n, k, device=DEV), gm.GraspState.zeros(1, m, n, k, DEV)
    W0, b0 = W.clone(), bias.clone()
    step(st, W, G)
    ad = gm.AdamWState.zeros([bias], 8)
    gm.AdamWStep(lr=1e-2)(ad, [bias], [gbias], clip=res)
    torch.cuda.synchronize()
    assert int(st.dev_status) == 0 and int(ad.step) == 1
    assert not torch.equal(W, W0)
    # from zero moments m / (1 - b1) = c g and sqrt(v / (1 - b2)) = c |g|, so the first step
    # moves an element by lr c g / (c |g| + eps): lr against the sign of its gradient, short
    # of it by lr eps / (c |g| + eps) (the gradients here are clipped to 1e-6 and below);
    # plus a dozen fp32 roundings
    move = (bias - b0).double() + 1e-2 * gbias.sign().double()
    short = 1e-8 / (float(res.scale) * gbias.double().abs() + 1e-8)
    assert bool((move.abs() <= 1e-2 * (short + 16 * U)).all())
    _check(gm, gm.mx4_quant(W, f), W.cpu(), fmt)


@pytest.mark.parametrize("M,N,K", [(5, 40, 300), (1, 300, 4100), (2048, 1500, 200)])
@pytest.mark.parametrize("ga,gb", [(1e20, 1e19), (3e30, 2e8), (1e-20, 1e-20), (1e-30, 1e-13), (1e25, 1e-25)])
def test_matrix_scales_whose_product_leaves_fp32(cuda_lib, M, N, K, ga, gb):
    """GM_NV4: the product of both gscale overflows, is subnormal, or is ordinary,
    while the sums times it lie in fp32's range. Entries are small beside the one that
    makes gscale, which meets zeros. An entry of D near fp32's end may be off by its
    last step, 2^-149; the exponent's halves multiply exactly otherwise."""
    gm = cuda_lib
    size = 0.02 if ga * gb > 1e30 else 300.0

    def operand(r, seed, gs, at, other):
        x = WL.random_matrix((1, r, K), seed).double().clamp(-4, 4) * size
        x[:, :, other] = 0
        x[:, :, at] = 0
        x[0, 0, at] = 2688.0
        x[0, -1] *= 1.0 if r == 1 else 0.0            # a row of zeros
        return gm.mx4_quant((x * gs).float().to(DEV), gm.GM_NV4)
    A, Bm = operand(M, 1, ga, 3, 40), operand(N, 2, gb, 40, 3)
    a, b = _values(gm, A).to(DEV), _values(gm, Bm).to(DEV)
    want, S = a @ b.transpose(-1, -2), a.abs() @ b.abs().transpose(-1, -2)
    assert float(want.abs().max()) < 1.6e38
    D = gm.mx4_matmul(A, Bm, out_dtype=F32)
    tol = (math.ceil(K / 64) + 2) * 2.0 ** -22 * S + U * want.abs() + 2.0 ** -149
    assert bool(((D.double() - want).abs() <= tol).all())
    gm.mx4_matmul(A, Bm, out=D, accumulate=True)
    assert bool(((D.double() - 2 * want).abs() <= 2 * tol + 2 * U * want.abs()).all())
