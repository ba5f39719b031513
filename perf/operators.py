"""Work that is timed of the AdamW step and the microscaled 4-bit operators.

``run`` computes each operator in plain torch (``own`` false) or through the
library's binding (``own`` true). Formulas:

* AdamW (t the steps done before this one, plus one):
  m <- b1 m + (1 - b1) g, v <- b2 v + (1 - b2) g^2,
  p <- (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps),
  g first scaled by the clip factor min(1, max_norm / (norm + 1e-6)) where the
  case clips; a NaN or infinity in the gradients then leaves everything as it was.
* 8-bit states: groups of 128 elements of a tensor. m: e4m3 codes of m / sm,
  sm = max(max|m| / 448, 2^-126). v: its root r as codes of r / sv with four
  exponent and four mantissa bits (no sign, largest 1.9375, code 1 at least
  where v is not zero in fp32), sv = max(max r / 1.9375, 2^-126). The codes are
  those of the unrounded m and r, so their plain form is computed in 64 bits.
* Microscaled 4 bits, e2m1 elements along a row: "mx" has blocks of 32 with a
  power-of-two scale 2^(floor(log2 max|x|) - 2); "nv" has blocks of 16 with an
  e4m3 scale rn(max|x| / (6 gs)) under a matrix scale gs = max|X| / 2688.
* Products D = A B^T of the values the codes stand for.
"""

import math

import torch

own = False

DEV = "cuda"
GROUP = 128
LR, BETA1, BETA2, EPS, WD = 1e-3, 0.9, 0.999, 1e-8, 0.1
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = {"mx": 32, "nv": 16}

# Shape groups (rows, columns, count) of the repository's parameter sets.
SETS = {
    "llama130m": ((768, 768, 48), (2048, 768, 24), (768, 2048, 12)),
    "llama1.1b": ((2048, 2048, 44), (256, 2048, 44), (5632, 2048, 44), (2048, 5632, 22)),
}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the norm weights of a 12-layer model of width 768: many tiny tensors, one call (latency)
        {"name": "adamw32-vectors", "op": "adamw", "bits": 32, "sizes": "25x768", "p": "f32",
         "g": "f32", "copy": "", "clip": False, "bad": False},
        # the LLaMA-130M-shaped set trained by AdamW alone (the comparison a Muon run is held to),
        # bf16 gradients clipped by their global norm, a bf16 working copy for the next forward
        {"name": "adamw32-set-clip", "op": "adamw", "bits": 32, "sizes": "llama130m", "p": "f32",
         "g": "bf16", "copy": "bf16", "clip": True, "bad": False},
        # the LLaMA-1.1B-shaped set: the largest step
        {"name": "adamw32-large-set", "op": "adamw", "bits": 32, "sizes": "llama1.1b", "p": "f32",
         "g": "bf16", "copy": "", "clip": False, "bad": False},
        # a few tensors of odd lengths, 16-bit weights without a master copy, 8-bit states
        {"name": "adamw8-odd", "op": "adamw", "bits": 8, "sizes": "1,7,129,1000,4097,65537,1000003",
         "p": "bf16", "g": "bf16", "copy": "", "clip": False, "bad": False},
        # an embedding table and an output head: what Muon leaves to AdamW, 8-bit states
        {"name": "adamw8-table-clip", "op": "adamw", "bits": 8, "sizes": "102402048,102402048,2048",
         "p": "f32", "g": "bf16", "copy": "bf16", "clip": True, "bad": False},
        # one token's activations before a decoding product (latency)
        {"name": "quant-mx-token", "op": "quant", "fmt": "mx", "batch": 1, "rows": 1, "cols": 3584,
         "x": "bf16", "both": False},
        # a training batch's activations, both orientations, columns not a multiple of the block
        {"name": "quant-mx-acts", "op": "quant", "fmt": "mx", "batch": 1, "rows": 4095, "cols": 2050,
         "x": "bf16", "both": True},
        # the updated fp32 weights of two Qwen2.5-7B MLP matrices, both orientations
        {"name": "quant-nv-weights", "op": "quant", "fmt": "nv", "batch": 2, "rows": 18944,
         "cols": 3584, "x": "f32", "both": True},
        # decoding: one token against a weight quantised once
        {"name": "product-mx-token", "op": "product", "fmt": "mx", "batch": 1, "rows": 1,
         "outs": 3584, "cols": 18944, "x": "bf16", "d": "bf16"},
        # a ragged batch of tokens, odd sizes
        {"name": "product-nv-odd", "op": "product", "fmt": "nv", "batch": 1, "rows": 1001,
         "outs": 2053, "cols": 771, "x": "f16", "d": "f16"},
        # a prefill batch against an MLP weight: the largest product
        {"name": "product-mx-large", "op": "product", "fmt": "mx", "batch": 1, "rows": 8192,
         "outs": 18944, "cols": 3584, "x": "bf16", "d": "bf16"},
        # a linear layer's training step: quantise X, W, dY both ways, forward, data and weight gradient
        {"name": "linear-nv-train", "op": "linear", "fmt": "nv", "rows": 4096, "outs": 5632,
         "cols": 2048, "x": "bf16", "d": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "quant", "product", "linear"])
    if op == "adamw":
        bits = rng.choice([32, 8])
        total = _log_int(rng, 1, 2 * 10 ** 8)
        count = min(_log_int(rng, 1, 600), total)
        cuts = sorted(rng.random() for _ in range(count - 1))
        edges = [0.0] + cuts + [1.0]
        sizes = [max(1, int(total * (b - a))) for a, b in zip(edges, edges[1:])]
        p = rng.choice(["f32", "f32", "bf16", "f16"])
        return {"op": "adamw", "bits": bits, "sizes": ",".join(str(s) for s in sizes), "p": p,
                "g": rng.choice(["f32", "bf16", "f16"]),
                "copy": rng.choice(["", "bf16", "f16"]) if p == "f32" else "",
                "clip": rng.random() < 0.5, "bad": rng.random() < 0.15}
    fmt = rng.choice(["mx", "nv"])
    x = rng.choice(["bf16", "f32", "f16"])
    if op == "quant":
        batch = rng.choice([1, 1, 2, 3])
        cols = _log_int(rng, 1, 20000)
        rows = _log_int(rng, 1, min(40000, 10 ** 8 // (batch * cols)))
        return {"op": "quant", "fmt": fmt, "batch": batch, "rows": rows, "cols": cols, "x": x,
                "both": rng.random() < 0.5}
    if op == "product":
        rows, outs = _log_int(rng, 1, 8192), _log_int(rng, 1, 10000)
        cols = _log_int(rng, 1, min(10000, 4 * 10 ** 11 // (rows * outs)))
        return {"op": "product", "fmt": fmt, "batch": rng.choice([1, 1, 1, 3]) if rows * outs < 10 ** 7 else 1,
                "rows": rows, "outs": outs, "cols": cols, "x": x, "d": rng.choice(["bf16", "f16", "f32"])}
    rows, outs = _log_int(rng, 1, 8192), _log_int(rng, 16, 6000)
    cols = _log_int(rng, 16, min(6000, 10 ** 11 // (rows * outs)))
    return {"op": "linear", "fmt": fmt, "rows": rows, "outs": outs, "cols": cols,
            "x": rng.choice(["bf16", "f16"]), "d": rng.choice(["bf16", "f16"])}


def _sizes(case):
    s = case["sizes"]
    if s in SETS:
        return [r * c for r, c, n in SETS[s] for _ in range(n)]
    if "x" in s:
        n, each = s.split("x")
        return [int(each)] * int(n)
    return [int(v) for v in s.split(",")]


# -------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(shape, g, dtype):
    """Gaussian values with a few large columns, as a transformer's activations have."""
    x = _randn(shape, g)
    cols = shape[-1]
    hot = torch.randint(0, cols, (max(1, cols // 256),), generator=g, device=DEV)
    x[..., hot] *= 20.0
    return x.to(dtype)


def _arena(sizes, dtype, per=1):
    """One buffer holding a tensor per size, each on a 256-byte boundary (as a
    program that allocates its optimizer's tensors together has them), and the views."""
    at, spans = 0, []
    for n in sizes:
        n = -(-n // per)
        spans.append((at, n))
        at += -(-n // 256) * 256
    flat = torch.zeros(at, dtype=dtype, device=DEV)
    return flat, [flat[a:a + n] for a, n in spans]


def _prepare_adamw(case, g, step):
    sizes = _sizes(case)
    small = case["bits"] == 8
    st = {"case": case, "flat": {}, "keep": {}, "copies": None, "mscale": [], "vscale": [],
          "step": torch.full((1,), step, dtype=torch.int64, device=DEV)}
    kept = torch.uint8 if small else torch.float32
    arenas = [("params", DT[case["p"]], 1), ("grads", DT[case["g"]], 1), ("m", kept, 1), ("v", kept, 1)]
    if case["copy"]:
        arenas.append(("copies", DT[case["copy"]], 1))
    if small:
        arenas += [("mscale", torch.float32, GROUP), ("vscale", torch.float32, GROUP),
                   ("m32", torch.float32, 1), ("v32", torch.float32, 1)]
    for name, dtype, per in arenas:
        st["flat"][name], st[name] = _arena(sizes, dtype, per)
    for i, n in enumerate(sizes):
        st["params"][i].copy_(0.02 * _randn((n,), g))
        st["grads"][i].copy_(1e-3 * _randn((n,), g))
        m = 1e-4 * _randn((n,), g)
        v = (1e-3 * _randn((n,), g)).square() * 0.3 + 1e-10
        state = zip(("m", "mscale", "v", "vscale"), _pack8(m.double(), v.double())) if small \
            else (("m", m), ("v", v))
        for name, value in state:
            st[name][i].copy_(value)
        if case["copy"]:
            st["copies"][i].copy_(st["params"][i])
    if case["bad"]:
        worst = max(st["grads"], key=lambda t: t.numel())
        worst[worst.numel() // 2] = float("inf")
    return st


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "adamw":
        return _prepare_adamw(case, g, 100 + seed % 7)
    if op == "quant":
        shape = (case["batch"], case["rows"], case["cols"])
        return {"case": case, "x": _activations(shape, g, DT[case["x"]])}
    if op == "product":
        x = _activations((case["batch"], case["rows"], case["cols"]), g, DT[case["x"]])
        w = 0.02 * _randn((case["batch"], case["outs"], case["cols"]), g)
        return {"case": case, "x": x, "w": _operand(w, case["fmt"])}
    return {"case": case, "x": _activations((1, case["rows"], case["cols"]), g, DT[case["x"]]),
            "w": 0.02 * _randn((1, case["outs"], case["cols"]), g),
            "dy": (1e-2 * _randn((1, case["rows"], case["outs"]), g)).to(DT[case["x"]])}


# ------------------------------------------------------------ 8-bit states
def _exponent(a, least):
    """floor(log2 a) of a >= 0 in 64 bits, at least `least`."""
    return ((a.view(torch.int64) >> 52) - 1023).clamp_min(least)


def _pow2(e):
    return ((e + 1023) << 52).view(torch.float64)


def _pack8(m, v):
    """Codes and group scales of m and v (flat, 64 bits)."""
    n = m.numel()
    pad = (-n) % GROUP
    mp = torch.nn.functional.pad(m, (0, pad)).view(-1, GROUP)
    vp = torch.nn.functional.pad(v, (0, pad)).view(-1, GROUP)
    rp = vp.sqrt()
    sm = (mp.abs().amax(1) / 448.0).clamp_min(2.0 ** -126)
    sv = (rp.amax(1) / 1.9375).clamp_min(2.0 ** -126)
    # a code counts steps of 2^-3 (e4m3, exponents from -6) or 2^-4 (exponents
    # from -14) of the value's power of two, above the steps of the lower ones
    y = (mp / sm[:, None]).clamp(-448.0, 448.0)
    e = _exponent(y.abs(), -6)
    k = (y.abs() * _pow2(3 - e)).round().to(torch.int64)
    cm = (((e + 6) << 3) + k) | ((y < 0).to(torch.int64) << 7)
    y = rp / sv[:, None]
    e = _exponent(y, -14)
    k = (y * _pow2(4 - e)).round().to(torch.int64)
    cv = (((e + 14) << 4) + k).clamp_max(255)
    cv = torch.maximum(cv, (vp.float() > 0).to(torch.int64))
    flat = lambda c: c.to(torch.uint8).reshape(-1)[:n]                    # noqa: E731
    return flat(cm), sm.float(), flat(cv), sv.float()


def _unpack8(cm, sm, cv, sv):
    """m and v of codes and group scales, 64 bits."""
    n = cm.numel()
    wide = lambda s: s.double().repeat_interleave(GROUP)[:n]              # noqa: E731
    m = cm.view(torch.float8_e4m3fn).double() * wide(sm)
    c = cv.to(torch.int64)
    e = (c >> 4).clamp_min(1)
    r = (c - ((e - 1) << 4)).double() * _pow2(e - 19) * wide(sv)
    return m, r * r


# --------------------------------------------------- microscaled 4-bit values
def _blocks(x, block):
    pad = (-x.shape[-1]) % 128
    x = torch.nn.functional.pad(x.float(), (0, pad))
    return x.view(*x.shape[:-1], -1, block)


def _scales(xb, fmt):
    """Stored scale bytes, their values in 64 bits, and the matrix scale (None for mx)."""
    top = xb.abs().amax(-1)
    if fmt == "mx":
        e = (top.view(torch.int32) >> 23) & 255
        byte = torch.where(e == 255, 255, (e - 2).clamp_min(0))
        val = _pow2(byte.to(torch.int64) - 127)
        return byte.to(torch.uint8), torch.where(byte == 255, math.nan, val), None
    gs = (top.amax((-1, -2)).double() / 2688.0).float()
    gs = torch.where(torch.isfinite(gs), gs, math.nan)
    t = top.double() / (6.0 * gs.double()[:, None, None])
    t = torch.where(gs[:, None, None] > 0, t, 0.0)
    step = _pow2(_exponent(t, -6) - 3)
    sb = ((t / step).round() * step).clamp_max(448.0)
    return sb.float().to(torch.float8_e4m3fn).view(torch.uint8), sb, gs


def _codes(xb, val, gs):
    """4-bit codes (sign in bit 3) of blocks under scales in 64 bits."""
    s = val if gs is None else val * gs.double()[:, None, None]
    a = torch.where((s > 0)[..., None], xb.double().abs() / s[..., None], 0.0)
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5.0
    return c | ((xb < 0) & (c > 0)).to(torch.uint8) << 3


def _operand(x, fmt):
    """A weight quantised once, as a program keeps it: packed codes, scales in
    the product's layout, the matrix scale."""
    xb = _blocks(x, BLOCK[fmt])
    byte, val, gs = _scales(xb, fmt)
    c = _codes(xb, val, gs).flatten(-2)
    B, rows, nb = byte.shape
    tiled = torch.nn.functional.pad(byte, (0, 0, 0, (-rows) % 128))
    tiled = tiled.view(B, -1, 4, 32, nb // 4, 4).permute(0, 1, 4, 3, 2, 5).contiguous()
    return {"codes": (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), "scales": tiled, "gs": gs,
            "rows": rows, "cols": x.shape[-1]}


def _e2m1():
    mag = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(mag + [-v for v in mag], device=DEV)


def _operand_values(q, fmt):
    c = torch.stack((q["codes"] & 15, q["codes"] >> 4), -1).flatten(-2)
    B, rows = c.shape[:2]
    byte = q["scales"].permute(0, 1, 4, 3, 2, 5).reshape(B, -1, q["scales"].shape[2] * 4)[:, :rows]
    if fmt == "mx":
        s = _pow2(byte.to(torch.int64) - 127).float()
    else:
        s = byte.contiguous().view(torch.float8_e4m3fn).float()
    x = (_e2m1()[c.int()].view(B, rows, -1, BLOCK[fmt]) * s[..., None]).flatten(-2)
    if q["gs"] is not None:
        x = x * q["gs"][:, None, None]
    return x[..., :q["cols"]]


def _values(x, fmt):
    """What the codes of x (along its last axis) stand for, fp32."""
    xb = _blocks(x, BLOCK[fmt])
    _, val, gs = _scales(xb, fmt)
    y = _e2m1()[_codes(xb, val, gs).int()] * val.float()[..., None]
    if gs is not None:
        y = y * gs[:, None, None, None]
    return y.flatten(-2)[..., :x.shape[-1]]


# --------------------------------------------------------------- plain forms
def _adamw_plain(st):
    case = st["case"]
    c, ok, norm = None, None, None
    if case["clip"]:
        norm = sum(g.double().square().sum() for g in st["grads"]).sqrt()
        ok = torch.isfinite(norm)
        c = (1.0 / (norm + 1e-6)).clamp_max(1.0)
    t = (st["step"] + 1).double()
    bc1, bc2 = 1 - BETA1 ** t, 1 - BETA2 ** t
    wide = torch.float64 if case["bits"] == 8 else torch.float32
    scale, root = (LR / bc1).to(wide), bc2.rsqrt().to(wide)
    keep = (lambda new, old: new) if ok is None else (lambda new, old: torch.where(ok, new, old))
    for i, p in enumerate(st["params"]):
        g = st["grads"][i].to(wide)
        if c is not None:
            g = g * c.to(wide)
        if case["bits"] == 8:
            m, v = _unpack8(st["m"][i], st["mscale"][i], st["v"][i], st["vscale"][i])
        else:
            m, v = st["m"][i], st["v"][i]
        m = m * BETA1 + g * (1 - BETA1)
        v = v * BETA2 + g * g * (1 - BETA2)
        new = p.to(wide) * (1 - LR * WD) - m / (v.sqrt() * root + EPS) * scale
        p.copy_(keep(new.to(p.dtype), p))
        if case["copy"]:
            st["copies"][i].copy_(keep(new.to(DT[case["copy"]]), st["copies"][i]))
        if case["bits"] == 8:
            for name, value in zip(("m", "mscale", "v", "vscale"), _pack8(m, v)):
                st[name][i].copy_(keep(value, st[name][i]))
            m, v = _unpack8(st["m"][i], st["mscale"][i], st["v"][i], st["vscale"][i])
            st["m32"][i].copy_(m)
            st["v32"][i].copy_(v)
        else:
            st["m"][i].copy_(keep(m, st["m"][i]))
            st["v"][i].copy_(keep(v, st["v"][i]))
    st["step"].add_(1 if ok is None else ok.to(torch.int64))
    return _adamw_outputs(st, norm)


def _adamw_outputs(st, norm):
    names = ("m32", "v32") if st["case"]["bits"] == 8 else ("m", "v")
    out = {"params": st["flat"]["params"], "m": st["flat"][names[0]], "v": st["flat"][names[1]],
           "step": st["step"]}
    if st["copies"] is not None:
        out["copies"] = st["flat"]["copies"]
    if norm is not None:
        out["norm"] = norm.view(1).float()
    return out


def _matmul_t(a, b, dtype):
    return torch.matmul(a, b.transpose(-1, -2)).to(dtype)


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "adamw":
        return _adamw_plain(st)
    fmt = case["fmt"]
    if op == "quant":
        if case["both"]:
            return [_values(st["x"], fmt), _values(st["x"].transpose(-1, -2), fmt)]
        return [_values(st["x"], fmt)]
    if op == "product":
        return _matmul_t(_values(st["x"], fmt), _operand_values(st["w"], fmt), DT[case["d"]])
    both = lambda t: (_values(t, fmt), _values(t.transpose(-1, -2), fmt))   # noqa: E731
    (x, xt), (w, wt), (dy, dyt) = both(st["x"]), both(st["w"]), both(st["dy"])
    return {"y": _matmul_t(x, w, DT[case["d"]]), "dx": _matmul_t(dy, wt, DT[case["d"]]),
            "dw": _matmul_t(dyt, xt, torch.float32)}


# ------------------------------------------------------- the library's calls
def _own(st):
    from bit_muon_optimizer_b200 import gmuon as gm
    case = st["case"]
    op = case["op"]
    if op == "adamw":
        keep = st["keep"]
        if not keep:
            keep["step"] = gm.AdamWStep(lr=LR, betas=(BETA1, BETA2), eps=EPS, wd=WD)
            keep["state"] = gm.AdamWState(case["bits"], st["m"], st["v"], st["mscale"], st["vscale"],
                                          st["step"])
        clip = gm.grad_norm(st["grads"], 1.0) if case["clip"] else None
        keep["step"](keep["state"], st["params"], st["grads"], copies=st["copies"], clip=clip)
        if case["bits"] == 8:
            keep["state"].moments(out=(st["m32"], st["v32"]))
        return _adamw_outputs(st, clip.norm if clip else None)
    fmt = gm.GM_MX4 if case["fmt"] == "mx" else gm.GM_NV4
    if op == "quant":
        if case["both"]:
            return [gm.mx4_dequant(q) for q in gm.mx4_quant(st["x"], fmt, cols=True)]
        return [gm.mx4_dequant(gm.mx4_quant(st["x"], fmt))]
    if op == "product":
        w = st["w"]
        W = gm.Mx4(fmt, w["rows"], w["cols"], w["codes"], w["scales"], w["gs"])
        return gm.mx4_matmul(gm.mx4_quant(st["x"], fmt), W, out_dtype=DT[case["d"]])
    d = DT[case["d"]]
    X, XT = gm.mx4_quant(st["x"], fmt, cols=True)
    W, WT = gm.mx4_quant(st["w"], fmt, cols=True)
    Y = gm.mx4_matmul(X, W, out_dtype=d)
    DY, DYT = gm.mx4_quant(st["dy"], fmt, cols=True)
    return {"y": Y, "dx": gm.mx4_matmul(DY, WT, out_dtype=d),
            "dw": gm.mx4_matmul(DYT, XT, out_dtype=torch.float32)}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- definition
def _exact_round(a, levels):
    """The level nearest to each |a| (fp64), ties to the even place in the list."""
    best = torch.full_like(a, math.inf)
    out = torch.zeros_like(a)
    for i, level in enumerate(levels):
        d = (a.abs() - level).abs()
        better = (d < best) | ((d == best) & (i % 2 == 0))
        best = torch.where(better, d, best)
        out = torch.where(better, level, out)
    return out * torch.sign(a)


_POWERS = [2.0 ** e for e in range(-200, 200)]


def _two_to(e):
    """2^e from a table (a library's power may be off in the last place)."""
    return torch.tensor(_POWERS, dtype=torch.float64, device=DEV)[(e + 200).clamp(0, 399).long()]


def _exact_float(x, mant, emin, top):
    """|x| rounded to `mant` fraction bits, exponents from emin, at most top (fp64)."""
    _, e = torch.frexp(x)
    ulp = _two_to((e - 1).clamp_min(emin) - mant)
    return torch.clamp(torch.round(x / ulp) * ulp, max=top)


def _exact_values(x, fmt):
    n = x.shape[-1]
    block = BLOCK[fmt]
    x = torch.nn.functional.pad(x.double(), (0, (-n) % block))
    xb = x.unflatten(-1, (-1, block))
    top = xb.abs().amax(-1, keepdim=True)
    if fmt == "mx":
        _, e = torch.frexp(top)
        s = _two_to((e - 3).clamp_min(-127))
        s = torch.where(torch.isfinite(top), s, math.nan)
    else:
        g = (x.abs().amax((-1, -2), keepdim=True) / 2688.0).float().double()[..., None]
        g = torch.where(torch.isfinite(g), g, math.nan)
        t = torch.where(g > 0, top / (6.0 * g), 0.0)
        s = _exact_float(t, 3, -6, 448.0) * g
    z = torch.where(s > 0, xb / s, 0.0)
    return (_exact_round(z, [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]) * s).flatten(-2)[..., :n]


def _exact_state8(m, v):
    """What 8 bits keep of m and v (the scales are kept in 32 bits)."""
    n = m.numel()
    grp = lambda t: torch.nn.functional.pad(t, (0, (-n) % GROUP)).view(-1, GROUP)   # noqa: E731
    mg, rg = grp(m), grp(v).sqrt()
    sm = (mg.abs().amax(1, keepdim=True) / 448.0).clamp_min(2.0 ** -126)
    sv = (rg.amax(1, keepdim=True) / 1.9375).clamp_min(2.0 ** -126)
    m8 = torch.sign(mg) * _exact_float(mg.abs() / sm, 3, -6, 448.0) * sm.float().double()
    r8 = _exact_float(rg / sv, 4, -14, 1.9375)
    r8 = torch.where((grp(v).float() > 0) & (r8 == 0), 2.0 ** -18, r8) * sv.float().double()
    return m8.flatten()[:n], r8.flatten()[:n].square()


def _exact_adamw(st):
    case = st["case"]
    sizes = _sizes(case)
    if sum(sizes) > 3 * 10 ** 8:
        return None
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in st["grads"]))
    skip = case["clip"] and not math.isfinite(norm)
    c = min(1.0, 1.0 / (norm + 1e-6)) if case["clip"] and not skip else 1.0
    t0 = int(st["step"][0])
    t = t0 + 1
    out = {"step": torch.tensor([t0 if skip else t], device=DEV)}
    views = {}
    for name in ("params", "m", "v") + (("copies",) if case["copy"] else ()):
        out[name], views[name] = _arena(sizes, torch.float64)
    if case["clip"]:
        out["norm"] = torch.tensor([norm], dtype=torch.float64, device=DEV)
    for i, p in enumerate(st["params"]):
        if case["bits"] == 8:
            at = torch.arange(p.numel(), device=DEV) // GROUP
            m = st["m"][i].view(torch.float8_e4m3fn).double() * st["mscale"][i].double()[at]
            e, f = (st["v"][i] >> 4).long(), (st["v"][i] & 15).double() / 16
            r = torch.where(e > 0, (1 + f) * _two_to(e - 15), f * 2.0 ** -14)
            v = (r * st["vscale"][i].double()[at]).square()
        else:
            m, v = st["m"][i].double(), st["v"][i].double()
        x = p.double()
        if not skip:
            g = st["grads"][i].double() * c
            m = BETA1 * m + (1 - BETA1) * g
            v = BETA2 * v + (1 - BETA2) * g.square()
            x = x - LR * (m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)).sqrt() + EPS) + WD * x)
            if case["bits"] == 8:
                m, v = _exact_state8(m, v)
        for name, value in (("params", x), ("m", m), ("v", v)):
            views[name][i].copy_(value)
        if case["copy"]:
            views["copies"][i].copy_(st["copies"][i] if skip else x)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "adamw":
        return _exact_adamw(st)
    fmt = case["fmt"]
    if op == "quant":
        out = [_exact_values(st["x"], fmt)]
        if case["both"]:
            out.append(_exact_values(st["x"].transpose(-1, -2), fmt))
        return out
    prod = lambda a, b: torch.matmul(a, b.transpose(-1, -2))               # noqa: E731
    if op == "product":
        g = _gen(seed)
        _activations((case["batch"], case["rows"], case["cols"]), g, DT[case["x"]])
        w = 0.02 * _randn((case["batch"], case["outs"], case["cols"]), g)
        return prod(_exact_values(st["x"], fmt), _exact_values(w, fmt))
    ev = lambda t: _exact_values(t, fmt)                                    # noqa: E731
    tr = lambda t: t.transpose(-1, -2)                                      # noqa: E731
    return {"y": prod(ev(st["x"]), ev(st["w"])), "dx": prod(ev(st["dy"]), ev(tr(st["w"]))),
            "dw": prod(ev(tr(st["dy"])), ev(tr(st["x"])))}


# ----------------------------------------------------------------------- work
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def work(case):
    op = case["op"]
    if op == "adamw":
        sizes = _sizes(case)
        n = sum(sizes)
        groups = sum(-(-s // GROUP) for s in sizes)
        per = 2 * _BYTES[case["p"]] + _BYTES[case["g"]] + (2 if case["copy"] else 0)
        # 8-bit states: codes in and out, and the moments handed back in fp32
        per += 16 if case["bits"] == 32 else 4 + 8
        scales = 0 if case["bits"] == 32 else groups * 16
        return {"bytes": n * per + scales, "flops": n * (18 if case["clip"] else 15)}
    block = BLOCK[case["fmt"]]
    x = _BYTES[case["x"]]
    if op == "quant":
        n = case["batch"] * case["rows"] * case["cols"]
        ways = 2 if case["both"] else 1
        return {"bytes": n * (x + 4 * ways), "flops": n * 3 * ways}
    rows, outs, cols = case["rows"], case["outs"], case["cols"]
    d = _BYTES[case["d"]]
    if op == "product":
        B = case["batch"]
        return {"bytes": int(B * (rows * cols * x + outs * cols * (0.5 + 1 / block) + rows * outs * d)),
                "flops": 2 * B * rows * outs * cols}
    return {"bytes": rows * cols * x + outs * cols * 4 + rows * outs * x
            + rows * outs * d + rows * cols * d + outs * cols * 4,
            "flops": 6 * rows * outs * cols}
