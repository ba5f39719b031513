"""Thin ctypes binding of libgmuon (include/gmuon.h).

Argument marshalling only: every step of the optimizer runs in the library's
CUDA kernels. Tensors are torch CUDA tensors, contiguous, batch-first
([B, rows, cols]); work is enqueued on torch's current CUDA stream. Importing
this module fails loudly when the library has not been built.
"""

from __future__ import annotations

import contextlib
import ctypes
import math
import os
import struct
from dataclasses import dataclass, field
from itertools import chain
from operator import attrgetter

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgmuon.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "gmuon.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m bit_muon_optimizer_b200.build`")
lib = ctypes.CDLL(LIB_PATH)

GM_OK, GM_E_ARG, GM_E_CUDA, GM_E_NONFINITE, GM_E_WORKSPACE, GM_E_UNSUPPORTED, GM_E_TIMEOUT = (
    0, -1, -2, -3, -4, -5, -6)
GM_F32, GM_BF16, GM_F16 = 0, 1, 2
GM_NS_STANDARD, GM_NS_GRAM = 0, 1
GM_OP_MOMENTUM_POWERIT, GM_OP_NEWTON_SCHULZ, GM_OP_GRAM_NS, GM_OP_GRASP_STEP = 1, 2, 3, 4
GM_MX4, GM_NV4 = 0, 1
GRID_BLOCK = 128

_DT = {torch.float32: GM_F32, torch.bfloat16: GM_BF16, torch.float16: GM_F16}

c_int, c_float, c_size_t, c_uint64, vp = (ctypes.c_int, ctypes.c_float, ctypes.c_size_t,
                                          ctypes.c_uint64, ctypes.c_void_p)


class GraspParams(ctypes.Structure):
    _fields_ = [("mu", c_float), ("eta", c_float), ("wd", c_float), ("k", c_int), ("T", c_int),
                ("ns", c_int), ("abc", ctypes.POINTER(c_float)),
                ("restart_after", ctypes.POINTER(c_int)), ("n_restart", c_int),
                ("eps", c_float), ("seed", c_uint64), ("power_steps", c_int),
                ("residual_from_codes", c_int), ("matrix_ids", vp), ("block", c_int)]


class GraspStateC(ctypes.Structure):
    _fields_ = [("codes4", vp), ("rscale", vp), ("cscale", vp), ("P8", vp), ("Pscale", vp),
                ("R8", vp), ("Rscale", vp), ("step", vp), ("dev_status", vp)]


class GraspWsLayout(ctypes.Structure):
    _fields_ = [("M", c_size_t), ("Q", c_size_t), ("P", c_size_t), ("R", c_size_t),
                ("X", c_size_t), ("scale", c_size_t), ("total", c_size_t)]


def _sig(name, res, args):
    f = getattr(lib, name)
    f.restype = res
    f.argtypes = args
    return f


_sig("gm_status_string", ctypes.c_char_p, [c_int])
_sig("gm_last_error", ctypes.c_char_p, [])
_sig("gm_version", c_int, [])
_sig("gm_workspace_bytes", c_size_t, [c_int, c_int, c_int, c_int, c_int, c_int])
_sig("gm_dequant_rebuild", c_int, [c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp, vp, vp, vp, vp])
_sig("gm_momentum_powerit", c_int, [c_int, c_int, c_int, c_int, c_float, vp, vp, c_int, vp,
                                    c_uint64, vp, vp, vp, vp, c_size_t, vp])
_sig("gm_grid_quant4", c_int, [c_int, c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp, vp, vp])
_sig("gm_quant8", c_int, [c_int, c_int, c_int, vp, vp, vp, vp])
_sig("gm_group_quant4", c_int, [c_int, c_int, c_int, vp, vp, vp, vp])
_sig("gm_group_dequant4", c_int, [c_int, c_int, c_int, vp, vp, vp, vp])
_sig("gm_mulaw_quant4", c_int, [c_int, c_int, c_int, c_float, vp, vp, vp, vp])
_sig("gm_mulaw_dequant4", c_int, [c_int, c_int, c_int, c_float, vp, vp, vp, vp])
_sig("gm_newton_schulz", c_int, [c_int, c_int, c_int, vp, c_int, vp, c_int, c_float, vp, c_int,
                                 vp, c_size_t, vp])
_sig("gm_newton_schulz_noalloc", c_int, [c_int, c_int, c_int, vp, c_int, vp, c_int, c_float, vp,
                                         c_int, vp])
_sig("gm_gram_ns", c_int, [c_int, c_int, c_int, vp, c_int, vp, c_int, vp, c_int, c_float, vp,
                           c_int, vp, c_size_t, vp])
_sig("gm_grasp_step", c_int, [c_int, c_int, c_int, ctypes.POINTER(GraspParams),
                              ctypes.POINTER(GraspStateC), vp, vp, c_int, vp, c_size_t, vp])
_sig("gm_grasp_state_update", c_int, [c_int, c_int, c_int, ctypes.POINTER(GraspParams),
                                      ctypes.POINTER(GraspStateC), vp, c_int, vp, c_size_t, vp])
_sig("gm_grasp_apply", c_int, [c_int, c_int, c_int, ctypes.POINTER(GraspParams),
                               ctypes.POINTER(GraspStateC), vp, vp, c_size_t, vp])
_sig("gm_grasp_orth", c_int, [c_int, c_int, c_int, ctypes.POINTER(GraspParams),
                              ctypes.POINTER(GraspStateC), vp, c_int, vp, c_size_t, vp])
_sig("gm_weight_update", c_int, [c_int, c_int, c_int, c_float, c_float, vp, c_int, vp, vp, c_int, vp])
_sig("gm_grasp_orth_peers", c_int, [c_int, c_int, c_int, ctypes.POINTER(GraspParams),
                                    ctypes.POINTER(GraspStateC), ctypes.POINTER(vp),
                                    ctypes.POINTER(vp), c_int, vp, c_int, vp, c_size_t, vp])


class IpcHandle(ctypes.Structure):
    _fields_ = [("bytes", ctypes.c_ubyte * 64)]


_sig("gm_ipc_export", c_int, [vp, ctypes.POINTER(IpcHandle), ctypes.POINTER(c_size_t)])
_sig("gm_ipc_open", c_int, [ctypes.POINTER(IpcHandle), ctypes.POINTER(vp)])
_sig("gm_ipc_close", c_int, [vp])
_sig("gm_grasp_workspace_layout", c_int, [c_int, c_int, c_int, c_int, c_int,
                                          ctypes.POINTER(GraspWsLayout)])
_sig("gm_ns_flops", c_int, [c_int, c_int, c_int, c_int, vp, c_int,
                            ctypes.POINTER(ctypes.c_double), ctypes.POINTER(c_int)])
_sig("gm_device_errors", c_int, [vp])
_sig("gm_test_wait_timeout", c_int, [vp, vp, ctypes.c_int64, vp])


class AdamWParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("wd", ctypes.c_double), ("bits", c_int), ("clip", vp),
                ("lr_dev", vp)]


ADAMW_SCRATCH_BYTES = 64
_sig("gm_grad_norm_workspace_bytes", c_size_t, [c_int])
_sig("gm_grad_norm", c_int, [c_int, vp, ctypes.c_double, vp, vp, vp, vp, c_size_t, vp])
_sig("gm_adamw_step", c_int, [c_int, vp, c_int, c_int, c_int, ctypes.POINTER(AdamWParams), vp, vp, vp, vp])
_sig("gm_adamw_step_mixed", c_int, [c_int, vp, vp, ctypes.POINTER(AdamWParams), vp, vp, vp, vp])
_sig("gm_adamw_begin", c_int, [ctypes.POINTER(AdamWParams), vp, vp, vp, vp])
_sig("gm_adamw_apply", c_int, [c_int, vp, c_int, c_int, c_int, ctypes.POINTER(AdamWParams), vp, vp])
_sig("gm_mx4_codes_bytes", c_size_t, [c_int, c_int, c_int])
_sig("gm_mx4_scales_bytes", c_size_t, [c_int, c_int, c_int, c_int])
_sig("gm_mx4_quant", c_int, [c_int, c_int, c_int, vp, c_int, ctypes.c_int64, ctypes.c_int64, c_int,
                             vp, vp, vp, vp, vp, vp])
_sig("gm_mx4_dequant", c_int, [c_int, c_int, c_int, c_int, vp, vp, vp, vp, c_int, vp])
_sig("gm_mx4_matmul", c_int, [c_int, c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp, vp, vp, c_int,
                              c_int, vp])
_sig("gm_adamw_unpack8", c_int, [c_int, vp, vp])


class GmuonError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib.gm_last_error().decode(errors="replace")
        super().__init__(f"{where}: {lib.gm_status_string(status).decode()} ({msg})")


def _check(status: int, where: str):
    if status != GM_OK:
        raise GmuonError(status, where)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _expect(t, shape, dtypes, name):
    """Checks the shape (a [m, n] matrix also stands for a batch of one) and
    dtype of a tensor handed to the library as a raw pointer."""
    shape = tuple(shape)
    got = tuple(t.shape)
    if got != shape and not (len(shape) >= 2 and shape[0] == 1 and got == shape[1:]):
        raise ValueError(f"{name}: expected shape {shape}, got {got}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} is not one of {tuple(dtypes)}")


def _ws_fits(ws, nbytes, name="ws"):
    """Checks that a caller-supplied workspace holds at least `nbytes`."""
    have = ws.numel() * ws.element_size()
    if have < nbytes:
        raise ValueError(f"{name}: {have} bytes, the call needs {nbytes}")


def _placed(tensors, names):
    """Checks that tensors are contiguous CUDA tensors."""
    for t, name in zip(tensors, names):
        if not t.is_cuda:
            raise ValueError(f"{name}: expected a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _bmn(X):
    if X.dim() == 2:
        return 1, X.shape[0], X.shape[1]
    if X.dim() != 3:
        raise ValueError("expected [B, m, n] or [m, n]")
    return X.shape[0], X.shape[1], X.shape[2]


def _floats(vals):
    if vals is None:
        return None
    arr = (c_float * len(vals))(*vals)
    return arr


def abc_table(abc, T):
    """Flatten a list of (a, b, c) triples (or None: constant quintic)."""
    if abc is None:
        return None
    flat = [float(v) for tri in abc for v in tri]
    if len(flat) != 3 * T:
        raise ValueError("abc must hold T triples")
    return _floats(flat)


_WS = {}


def workspace(nbytes: int, device=None, tag="default") -> torch.Tensor:
    """A cached 256-byte-aligned device scratch buffer of at least nbytes."""
    device = torch.device(device or torch.cuda.current_device())
    key = (tag, device)
    buf = _WS.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _WS[key] = buf
    return buf


def workspace_bytes(op, B, m, n, k=0, ns=GM_NS_STANDARD) -> int:
    return int(lib.gm_workspace_bytes(op, B, m, n, k, ns))


# ----------------------------------------------------------------- entry points

def dequant_rebuild(codes4, rscale, cscale, P8=None, Pscale=None, R8=None, Rscale=None, out=None):
    B, m, n2 = _bmn(codes4)
    n = 2 * n2
    k = 0 if P8 is None else P8.shape[-1]
    mb, nb = -(-m // GRID_BLOCK), -(-n // GRID_BLOCK)
    _expect(codes4, (B, m, n2), (torch.uint8,), "codes4")
    _expect(rscale, (B, m, nb), (torch.float32,), "rscale")
    _expect(cscale, (B, mb, n), (torch.float32,), "cscale")
    if k:
        _expect(P8, (B, m, k), (torch.int8,), "P8")
        _expect(Pscale, (B, k), (torch.float32,), "Pscale")
        _expect(R8, (B, n, k), (torch.int8,), "R8")
        _expect(Rscale, (B, k), (torch.float32,), "Rscale")
    if out is None:
        out = torch.empty((B, m, n), dtype=torch.float32, device=codes4.device)
    _expect(out, (B, m, n), (torch.float32,), "out")
    _check(lib.gm_dequant_rebuild(B, m, n, k, _ptr(codes4), _ptr(rscale), _ptr(cscale), _ptr(P8),
                                  _ptr(Pscale), _ptr(R8), _ptr(Rscale), _ptr(out), _stream()),
           "gm_dequant_rebuild")
    return out


def momentum_powerit(G, k, mu=0.95, M_prev=None, R_prev=None, seed=0):
    B, m, n = _bmn(G)
    _expect(G, (B, m, n), tuple(_DT), "G")
    if M_prev is not None:
        _expect(M_prev, (B, m, n), (torch.float32,), "M_prev")
    if R_prev is not None:
        _expect(R_prev, (B, n, k), (torch.float32,), "R_prev")
    dev = G.device
    M = torch.empty((B, m, n), dtype=torch.float32, device=dev)
    P = torch.empty((B, m, k), dtype=torch.float32, device=dev)
    R = torch.empty((B, n, k), dtype=torch.float32, device=dev)
    nb = workspace_bytes(GM_OP_MOMENTUM_POWERIT, B, m, n, k)
    ws = workspace(nb, dev)
    _check(lib.gm_momentum_powerit(B, m, n, k, mu, _ptr(M_prev), _ptr(G), _DT[G.dtype],
                                   _ptr(R_prev), seed, _ptr(M), _ptr(P), _ptr(R), _ptr(ws), nb,
                                   _stream()), "gm_momentum_powerit")
    return M, P, R


def grid_quant4(X, P=None, R=None, out=None):
    B, m, n = _bmn(X)
    dev = X.device
    k = 0 if P is None else P.shape[-1]
    _expect(X, (B, m, n), (torch.float32,), "X")
    if (P is None) != (R is None):
        raise ValueError("P and R must both be given or both be None")
    if k:
        _expect(P, (B, m, k), (torch.float32,), "P")
        _expect(R, (B, n, k), (torch.float32,), "R")
    if out is not None:
        codes, rs, cs = out
        _expect(codes, (B, m, n // 2), (torch.uint8,), "codes")
        _expect(rs, (B, m, -(-n // GRID_BLOCK)), (torch.float32,), "rscale")
        _expect(cs, (B, -(-m // GRID_BLOCK), n), (torch.float32,), "cscale")
    else:
        codes = torch.empty((B, m, n // 2), dtype=torch.uint8, device=dev)
        rs = torch.empty((B, m, -(-n // GRID_BLOCK)), dtype=torch.float32, device=dev)
        cs = torch.empty((B, -(-m // GRID_BLOCK), n), dtype=torch.float32, device=dev)
    _check(lib.gm_grid_quant4(B, m, n, GRID_BLOCK, k, _ptr(X), _ptr(P), _ptr(R), _ptr(codes), _ptr(rs),
                              _ptr(cs), _stream()), "gm_grid_quant4")
    return codes, rs, cs


def quant8(X):
    B, rows, k = _bmn(X)
    _expect(X, (B, rows, k), (torch.float32,), "X")
    codes = torch.empty((B, rows, k), dtype=torch.int8, device=X.device)
    scale = torch.empty((B, k), dtype=torch.float32, device=X.device)
    _check(lib.gm_quant8(B, rows, k, _ptr(X), _ptr(codes), _ptr(scale), _stream()), "gm_quant8")
    return codes, scale


GROUP = 128   # elements per scale of the 4bit-Muon-base codec


def group_quant4(X, out=None):
    """4bit-Muon-base codes of fp32 [B, m, n] (or [m, n]): (codes [B, m, n/2]
    uint8, scales [B, m n / 128] fp32)."""
    B, m, n = _bmn(X)
    _expect(X, (B, m, n), (torch.float32,), "X")
    if out is not None:
        codes, gs = out
    else:
        codes = torch.empty((B, m, n // 2), dtype=torch.uint8, device=X.device)
        gs = torch.empty((B, m * n // GROUP), dtype=torch.float32, device=X.device)
    _expect(codes, (B, m, n // 2), (torch.uint8,), "codes")
    _expect(gs, (B, m * n // GROUP), (torch.float32,), "gscale")
    _check(lib.gm_group_quant4(B, m, n, _ptr(X), _ptr(codes), _ptr(gs), _stream()),
           "gm_group_quant4")
    return codes, gs


def group_dequant4(codes, gscale, out=None):
    """fp32 [B, m, n] from 4bit-Muon-base codes and scales."""
    B, m, n2 = _bmn(codes)
    n = 2 * n2
    _expect(codes, (B, m, n2), (torch.uint8,), "codes")
    _expect(gscale, (B, m * n // GROUP), (torch.float32,), "gscale")
    if out is None:
        out = torch.empty((B, m, n), dtype=torch.float32, device=codes.device)
    _expect(out, (B, m, n), (torch.float32,), "out")
    _check(lib.gm_group_dequant4(B, m, n, _ptr(codes), _ptr(gscale), _ptr(out), _stream()),
           "gm_group_dequant4")
    return out


MULAW_MU = 255.0


def mulaw_quant4(X, mu=MULAW_MU, out=None):
    """MuonQ's mu-law 4-bit codes of fp32 [B, m, n] (or [m, n]), in the group
    layout of ``group_quant4``: (codes [B, m, n/2] uint8, scales [B, m n / 128])."""
    B, m, n = _bmn(X)
    _expect(X, (B, m, n), (torch.float32,), "X")
    if out is not None:
        codes, gs = out
    else:
        codes = torch.empty((B, m, n // 2), dtype=torch.uint8, device=X.device)
        gs = torch.empty((B, m * n // GROUP), dtype=torch.float32, device=X.device)
    _expect(codes, (B, m, n // 2), (torch.uint8,), "codes")
    _expect(gs, (B, m * n // GROUP), (torch.float32,), "gscale")
    _check(lib.gm_mulaw_quant4(B, m, n, float(mu), _ptr(X), _ptr(codes), _ptr(gs), _stream()),
           "gm_mulaw_quant4")
    return codes, gs


def mulaw_dequant4(codes, gscale, mu=MULAW_MU, out=None):
    """fp32 [B, m, n] from mu-law codes and group scales."""
    B, m, n2 = _bmn(codes)
    n = 2 * n2
    _expect(codes, (B, m, n2), (torch.uint8,), "codes")
    _expect(gscale, (B, m * n // GROUP), (torch.float32,), "gscale")
    if out is None:
        out = torch.empty((B, m, n), dtype=torch.float32, device=codes.device)
    _expect(out, (B, m, n), (torch.float32,), "out")
    _check(lib.gm_mulaw_dequant4(B, m, n, float(mu), _ptr(codes), _ptr(gscale), _ptr(out),
                                 _stream()), "gm_mulaw_dequant4")
    return out


def newton_schulz(X, abc=None, T=5, eps=1e-7, out_dtype=torch.float32, out=None, ws=None):
    B, m, n = _bmn(X)
    _expect(X, (B, m, n), tuple(_DT), "X")
    O = out if out is not None else torch.empty((B, m, n), dtype=out_dtype, device=X.device)
    _expect(O, (B, m, n), tuple(_DT), "out")
    out_dtype = O.dtype
    nb = workspace_bytes(GM_OP_NEWTON_SCHULZ, B, m, n)
    ws = ws if ws is not None else workspace(nb, X.device)
    _ws_fits(ws, nb)
    _check(lib.gm_newton_schulz(B, m, n, _ptr(X), _DT[X.dtype], abc_table(abc, T), T, eps,
                                _ptr(O), _DT[out_dtype], _ptr(ws), nb, _stream()),
           "gm_newton_schulz")
    return O


NOALLOC_SCRATCH_BYTES = 64 << 20


def newton_schulz_noalloc(X, abc=None, T=5, eps=1e-7, out_dtype=torch.float32, out=None):
    """gm_newton_schulz through the entry point that allocates no device memory
    (its scratch is a fixed 64 MiB array inside the library). ``out`` must be
    preallocated by callers that cannot allocate either."""
    B, m, n = _bmn(X)
    _expect(X, (B, m, n), tuple(_DT), "X")
    O = out if out is not None else torch.empty((B, m, n), dtype=out_dtype, device=X.device)
    _expect(O, (B, m, n), tuple(_DT), "out")
    _check(lib.gm_newton_schulz_noalloc(B, m, n, _ptr(X), _DT[X.dtype], abc_table(abc, T), T, eps,
                                        _ptr(O), _DT[O.dtype], _stream()),
           "gm_newton_schulz_noalloc")
    return O


def gram_ns(X, abc=None, T=5, restart_after=(2,), eps=1e-7, out_dtype=torch.float32, out=None,
            ws=None):
    B, m, n = _bmn(X)
    _expect(X, (B, m, n), tuple(_DT), "X")
    O = out if out is not None else torch.empty((B, m, n), dtype=out_dtype, device=X.device)
    _expect(O, (B, m, n), tuple(_DT), "out")
    out_dtype = O.dtype
    nb = workspace_bytes(GM_OP_GRAM_NS, B, m, n)
    ws = ws if ws is not None else workspace(nb, X.device)
    _ws_fits(ws, nb)
    rl = list(restart_after)
    rarr = (c_int * max(1, len(rl)))(*rl) if rl else None
    _check(lib.gm_gram_ns(B, m, n, _ptr(X), _DT[X.dtype], abc_table(abc, T), T, rarr, len(rl),
                          eps, _ptr(O), _DT[out_dtype], _ptr(ws), nb, _stream()), "gm_gram_ns")
    return O


_sig("gm_gram_ns_trace", c_int, [c_int, c_int, c_int, vp, c_int, vp, c_int, vp, c_int, c_float,
                                 vp, c_int, vp, vp, vp, c_size_t, vp])


def gram_ns_trace(X, abc=None, T=5, restart_after=(2,), eps=1e-7, out_dtype=torch.float32):
    """gm_gram_ns_trace: returns (O, R_trace, Q_trace), the traces fp16
    [T, B, N, N] (N = min(m, n)): Q_t after every step, R_t where the chain
    computes it (zeros at t = T; the restarted Gram after a restart step)."""
    B, m, n = _bmn(X)
    _expect(X, (B, m, n), tuple(_DT), "X")
    N = min(m, n)
    Np = -(-N // 64) * 64
    O = torch.empty((B, m, n), dtype=out_dtype, device=X.device)
    Rt = torch.zeros((T, B, Np, Np), dtype=torch.float16, device=X.device)
    Qt = torch.zeros_like(Rt)
    nb = workspace_bytes(GM_OP_GRAM_NS, B, m, n)
    ws = workspace(nb, X.device)
    rl = list(restart_after)
    rarr = (c_int * max(1, len(rl)))(*rl) if rl else None
    _check(lib.gm_gram_ns_trace(B, m, n, _ptr(X), _DT[X.dtype], abc_table(abc, T), T, rarr, len(rl),
                                eps, _ptr(O), _DT[out_dtype], _ptr(Rt), _ptr(Qt), _ptr(ws), nb,
                                _stream()), "gm_gram_ns_trace")
    return O, Rt[..., :N, :N], Qt[..., :N, :N]


def ns_flops(ns, m, n, T=5, restart_after=(2,)):
    rl = list(restart_after) if ns == GM_NS_GRAM else []
    rarr = (c_int * max(1, len(rl)))(*rl) if rl else None
    f = ctypes.c_double()
    cnt = c_int()
    _check(lib.gm_ns_flops(ns, m, n, T, rarr, len(rl), ctypes.byref(f), ctypes.byref(cnt)),
           "gm_ns_flops")
    return f.value, cnt.value


def device_errors():
    _check(lib.gm_device_errors(_stream()), "gm_device_errors")


def wait_timeout_probe(limit_ns=20_000_000):
    """gm_test_wait_timeout: one product launch whose bounded wait runs out
    after limit_ns (a test hook of the failure path)."""
    X = torch.zeros((256, 256), dtype=torch.bfloat16, device="cuda")
    D = torch.empty_like(X)
    _check(lib.gm_test_wait_timeout(_ptr(X), _ptr(D), int(limit_ns), _stream()),
           "gm_test_wait_timeout")
    return X, D


@dataclass
class GraspState:
    """Device tensors of the quantized momentum of B same-shape matrices."""
    codes4: torch.Tensor
    rscale: torch.Tensor
    cscale: torch.Tensor
    P8: torch.Tensor
    Pscale: torch.Tensor
    R8: torch.Tensor
    Rscale: torch.Tensor
    step: torch.Tensor
    dev_status: torch.Tensor

    @staticmethod
    def zeros(B, m, n, k, device=None):
        d = device or torch.device("cuda")
        mb, nb = -(-m // GRID_BLOCK), -(-n // GRID_BLOCK)
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=d)   # noqa: E731
        return GraspState(z((B, m, n // 2), torch.uint8), z((B, m, nb), torch.float32),
                          z((B, mb, n), torch.float32), z((B, m, k), torch.int8),
                          z((B, k), torch.float32), z((B, n, k), torch.int8),
                          z((B, k), torch.float32), z((1,), torch.int64), z((1,), torch.int32))

    def tensors(self):
        return [self.codes4, self.rscale, self.cscale, self.P8, self.Pscale, self.R8,
                self.Rscale, self.step, self.dev_status]

    def check(self, B, m, n, k):
        """Raises ValueError unless every tensor has the layout gm_grasp_step
        reads and writes for B matrices of m x n at top rank k."""
        mb, nb = -(-m // GRID_BLOCK), -(-n // GRID_BLOCK)
        f32, i8 = (torch.float32,), (torch.int8,)
        _expect(self.codes4, (B, m, n // 2), (torch.uint8,), "codes4")
        _expect(self.rscale, (B, m, nb), f32, "rscale")
        _expect(self.cscale, (B, mb, n), f32, "cscale")
        _expect(self.P8, (B, m, k), i8, "P8")
        _expect(self.Pscale, (B, k), f32, "Pscale")
        _expect(self.R8, (B, n, k), i8, "R8")
        _expect(self.Rscale, (B, k), f32, "Rscale")
        _expect(self.step, (1,), (torch.int64,), "step")
        _expect(self.dev_status, (1,), (torch.int32,), "dev_status")
        _placed(self.tensors(), ["codes4", "rscale", "cscale", "P8", "Pscale", "R8", "Rscale",
                                 "step", "dev_status"])

    def c_struct(self):
        return GraspStateC(*[t.data_ptr() for t in self.tensors()])

    def clone(self):
        return GraspState(*[t.clone() for t in self.tensors()])


def ipc_export(t):
    """(handle bytes, byte offset) of the device allocation holding tensor t (gm_ipc_export)."""
    _placed((t,), ("t",))
    h = IpcHandle()
    off = c_size_t()
    _check(lib.gm_ipc_export(_ptr(t), ctypes.byref(h), ctypes.byref(off)), "gm_ipc_export")
    return bytes(h.bytes), off.value


def ipc_open(handle: bytes) -> int:
    """Device address of the start of another process's exported allocation (gm_ipc_open)."""
    h = IpcHandle()
    ctypes.memmove(h.bytes, handle, 64)
    base = vp()
    _check(lib.gm_ipc_open(ctypes.byref(h), ctypes.byref(base)), "gm_ipc_open")
    return base.value


def ipc_close(base: int) -> None:
    _check(lib.gm_ipc_close(vp(base)), "gm_ipc_close")


def weight_update(W, O, eta, wd=0.0, skip=None):
    """W <- W - eta (O + wd W) in place (gm_weight_update); O in float32, bfloat16 or
    float16 of W's shape. ``skip`` (optional device int32): one flag for the batch
    ([1]) or one per matrix ([B]); a flagged matrix keeps its weights."""
    B, m, n = _bmn(W)
    _expect(W, (B, m, n), (torch.float32,), "W")
    _expect(O, (B, m, n), (torch.float32, torch.bfloat16, torch.float16), "O")
    stride = 0
    if skip is not None:
        if skip.dtype != torch.int32 or not skip.is_contiguous() or skip.numel() not in (1, B):
            raise ValueError("skip: a contiguous int32 tensor of 1 or B flags expected")
        stride = 0 if skip.numel() == 1 else 1
        _placed((W, O, skip), ("W", "O", "skip"))
    else:
        _placed((W, O), ("W", "O"))
    _check(lib.gm_weight_update(B, m, n, float(eta), float(wd), _ptr(O), _DT[O.dtype], _ptr(W),
                                _ptr(skip), stride, _stream()), "gm_weight_update")
    return W


class GraspStep:
    """Marshals one gm_grasp_step call for a fixed shape batch.

    ``matrix_ids`` (optional): each matrix's index in the whole parameter set,
    used by the Rademacher start vectors (default 0 .. B-1); ``power_steps``
    (1..3) and ``residual_from_codes`` select the ablation variants."""

    def __init__(self, B, m, n, k, mu=0.95, eta=0.02, wd=0.0, T=5, ns=GM_NS_STANDARD, abc=None,
                 restart_after=(2,), eps=1e-7, seed=0, device=None, ws=None, power_steps=1,
                 residual_from_codes=False, matrix_ids=None):
        self.B, self.m, self.n, self.k = B, m, n, k
        self._abc = abc_table(abc, T)
        rl = list(restart_after) if ns == GM_NS_GRAM else []
        self._rarr = (c_int * max(1, len(rl)))(*rl)
        dev = device or torch.device("cuda")
        self.ids = None
        if matrix_ids is not None:
            ids = [int(i) for i in matrix_ids]
            if len(ids) != B or not all(0 <= i < 65536 for i in ids):
                raise ValueError("matrix_ids: B indices in [0, 65536) expected")
            self.ids = torch.tensor(ids, dtype=torch.int64, device=dev)
        self.params = GraspParams(mu, eta, wd, k, T, ns,
                                  ctypes.cast(self._abc, ctypes.POINTER(c_float)) if self._abc else None,
                                  ctypes.cast(self._rarr, ctypes.POINTER(c_int)) if rl else None,
                                  len(rl), eps, seed, int(power_steps), int(bool(residual_from_codes)),
                                  self.ids.data_ptr() if self.ids is not None else None)
        self.ws_bytes = workspace_bytes(GM_OP_GRASP_STEP, B, m, n, k, ns)
        if ws is None:
            ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        self.ws = ws
        lay = GraspWsLayout()
        _check(lib.gm_grasp_workspace_layout(B, m, n, k, ns, ctypes.byref(lay)),
               "gm_grasp_workspace_layout")
        self.layout = lay
        self.ns = ns

    def __call__(self, state: GraspState, W, G):
        B, m, n = self.B, self.m, self.n
        _expect(W, (B, m, n), (torch.float32,), "W")
        _expect(G, (B, m, n), tuple(_DT), "G")
        state.check(B, m, n, self.k)
        _placed((W, G), ("W", "G"))
        _ws_fits(self.ws, self.ws_bytes)
        st = state.c_struct()
        _check(lib.gm_grasp_step(self.B, self.m, self.n, ctypes.byref(self.params), ctypes.byref(st),
                                 _ptr(W), _ptr(G), _DT[G.dtype], _ptr(self.ws), self.ws_bytes,
                                 _stream()), "gm_grasp_step")

    def state_update(self, state: GraspState, G):
        """Worked steps 1-5 alone (gm_grasp_state_update)."""
        B, m, n = self.B, self.m, self.n
        _expect(G, (B, m, n), tuple(_DT), "G")
        state.check(B, m, n, self.k)
        _placed((G,), ("G",))
        _ws_fits(self.ws, self.ws_bytes)
        st = state.c_struct()
        _check(lib.gm_grasp_state_update(B, m, n, ctypes.byref(self.params), ctypes.byref(st),
                                         _ptr(G), _DT[G.dtype], _ptr(self.ws), self.ws_bytes,
                                         _stream()), "gm_grasp_state_update")

    def apply(self, state: GraspState, W):
        """Worked step 6 alone (gm_grasp_apply) on the NS input the state update left."""
        B, m, n = self.B, self.m, self.n
        _expect(W, (B, m, n), (torch.float32,), "W")
        state.check(B, m, n, self.k)
        _placed((W,), ("W",))
        _ws_fits(self.ws, self.ws_bytes)
        st = state.c_struct()
        _check(lib.gm_grasp_apply(B, m, n, ctypes.byref(self.params), ctypes.byref(st), _ptr(W),
                                  _ptr(self.ws), self.ws_bytes, _stream()), "gm_grasp_apply")

    def orth(self, state: GraspState, out=None, dtype=torch.bfloat16):
        """Worked step 6 up to O = NS(M_t) (gm_grasp_orth) on the NS input the state
        update left; O [B, m, n] in ``dtype`` (float32, bfloat16 or float16), not
        written when the state update flagged a non-finite value."""
        B, m, n = self.B, self.m, self.n
        state.check(B, m, n, self.k)
        if out is None:
            out = torch.empty((B, m, n), dtype=dtype, device=self.ws.device)
        _expect(out, (B, m, n), (torch.float32, torch.bfloat16, torch.float16), "O")
        _placed((out,), ("O",))
        _ws_fits(self.ws, self.ws_bytes)
        st = state.c_struct()
        _check(lib.gm_grasp_orth(B, m, n, ctypes.byref(self.params), ctypes.byref(st), _ptr(out),
                                 _DT[out.dtype], _ptr(self.ws), self.ws_bytes, _stream()),
               "gm_grasp_orth")
        return out

    def orth_peers(self, state: GraspState, peer_O, peer_flags, dst_index, dtype=torch.bfloat16):
        """O = NS(M_t) on the NS input the state update left, stored into every receive
        buffer of ``peer_O`` (device addresses of [.][m][n] ``dtype`` buffers, this
        process's or mapped from others) at matrix dst_index[b], with the step's status
        in ``peer_flags`` (int32 buffers) at the same index (gm_grasp_orth_peers)."""
        B, m, n = self.B, self.m, self.n
        state.check(B, m, n, self.k)
        if not 1 <= len(peer_O) == len(peer_flags) <= 8:
            raise ValueError("1 to 8 receive buffers, one flag buffer each")
        if dst_index.dtype != torch.int64 or tuple(dst_index.shape) != (B,):
            raise ValueError("dst_index: int64 [B] expected")
        _placed((dst_index,), ("dst_index",))
        _ws_fits(self.ws, self.ws_bytes)
        po = (vp * len(peer_O))(*[vp(int(a)) for a in peer_O])
        pf = (vp * len(peer_flags))(*[vp(int(a)) for a in peer_flags])
        st = state.c_struct()
        _check(lib.gm_grasp_orth_peers(B, m, n, ctypes.byref(self.params), ctypes.byref(st), po, pf,
                                       len(peer_O), _ptr(dst_index), _DT[dtype], _ptr(self.ws),
                                       self.ws_bytes, _stream()), "gm_grasp_orth_peers")

    def direction(self, state: GraspState, G, out=None, dtype=torch.bfloat16):
        """Worked steps 1-5 and O = NS(M_t): the state update, then ``orth``."""
        self.state_update(state, G)
        return self.orth(state, out, dtype)

    # stage buffers inside the workspace (views; valid after the step ran)
    def _view(self, off, shape, dtype):
        nbytes = 1
        for s in shape:
            nbytes *= s
        nbytes *= torch.empty((), dtype=dtype).element_size()
        return self.ws[off:off + nbytes].view(dtype).view(shape)

    def stage_M(self):
        return self._view(self.layout.M, (self.B, self.m, self.n), torch.float32)

    def stage_Q(self):
        return self._view(self.layout.Q, (self.B, self.n, self.k), torch.float32)

    def stage_P(self):
        return self._view(self.layout.P, (self.B, self.m, self.k), torch.float32)

    def stage_R(self):
        return self._view(self.layout.R, (self.B, self.n, self.k), torch.float32)

    def stage_scale(self):
        return self._view(self.layout.scale, (self.B,), torch.float32)

    def stage_X(self):
        N, Mp = min(self.m, self.n), max(self.m, self.n)
        dt = torch.float16 if self.ns == GM_NS_GRAM else torch.bfloat16
        return self._view(self.layout.X, (self.B, N, Mp), dt)


# ------------------------------------------------- AdamW over lists of tensors

_HERE = contextlib.nullcontext()
_numel, _get_device, _is_contiguous, _data_ptr, _dtype = (
    torch.Tensor.numel, torch.Tensor.get_device, torch.Tensor.is_contiguous, torch.Tensor.data_ptr,
    attrgetter("dtype"))


def _on(device):
    """The library works on the current device: makes `device` that, where it is not."""
    if device.index == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(device)


def _stream_of(device):
    """The address of torch's current stream on `device` (a stream object costs 3 us)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _list_of(tensors, name, dtypes, device=None, numels=None):
    """Checks a list of non-empty contiguous CUDA tensors on one device; returns the
    device, the element counts and the set of dtypes."""
    if not isinstance(tensors, (list, tuple)) or not tensors:
        raise ValueError(f"{name}: a non-empty list of tensors expected")
    dev = tensors[0].device if device is None else device
    # whole lists at a time: a loop with messages costs a small step more than its kernels
    counts = list(map(_numel, tensors))
    kinds = set(map(_dtype, tensors))
    if not (dev.type == "cuda" and set(map(_get_device, tensors)) == {dev.index} and kinds <= dtypes
            and all(map(_is_contiguous, tensors))
            and (0 not in counts if numels is None else counts == numels)):
        _list_error(tensors, name, dtypes, dev, numels)
    return dev, counts, kinds


def _list_error(tensors, name, dtypes, dev, numels):
    """The first thing wrong with a list that _list_of refuses."""
    if numels is not None and len(tensors) != len(numels):
        raise ValueError(f"{name}: expected {len(numels)} tensors, got {len(tensors)}")
    for i, t in enumerate(tensors):
        if t.dtype not in dtypes:
            raise ValueError(f"{name}[{i}]: dtype {t.dtype} is not one of {tuple(dtypes)}")
        n = t.numel()
        if n == 0 if numels is None else n != numels[i]:
            raise ValueError(f"{name}[{i}]: {n} elements"
                             + ("" if numels is None else f", expected {numels[i]}"))
        if not t.is_cuda:
            raise ValueError(f"{name}[{i}]: expected a CUDA tensor")
        if t.device != dev:
            raise ValueError(f"{name}[{i}]: on {t.device}, expected on {dev}")
        if not t.is_contiguous():
            raise ValueError(f"{name}[{i}]: expected a contiguous tensor")
    raise ValueError(f"{name}: expected CUDA tensors, got {dev}")


_FLOATS = frozenset(_DT)
_F32 = frozenset((torch.float32,))
_U8 = frozenset((torch.uint8,))


def _rows(*columns):
    """A host table of int64 rows for the library: entry i of every column."""
    return struct.pack(f"{len(columns) * len(columns[0])}q", *chain.from_iterable(zip(*columns)))


def _addresses(tensors):
    return list(map(_data_ptr, tensors))


def _scalar(t, dtype, name, device):
    """Checks a one-element tensor whose address goes to the library."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.numel() != 1:
        raise ValueError(f"{name}: expected a one-element {dtype} tensor")
    if t.device != device:
        raise ValueError(f"{name}: expected on {device}, got {t.device}")


@dataclass
class GradNorm:
    """The result of ``grad_norm``, on the device: ``norm`` f32 [1], ``scale`` f64
    [1] (the clip factor), ``status`` int32 [1] (GM_E_NONFINITE when a gradient
    holds a NaN or infinity), and the call's workspace. ``AdamWStep`` takes the
    whole, ``weight_update`` the status as its skip flag."""
    norm: torch.Tensor
    scale: torch.Tensor
    status: torch.Tensor
    ws: torch.Tensor


def grad_norm(grads, max_norm=None, out=None) -> GradNorm:
    """Norm over all elements of a list of gradients (fp32, bf16, fp16, mixed), and
    min(1, max_norm / (norm + 1e-6)) (1 without ``max_norm``). ``out``: an earlier
    result of a list of at most this length, to write into."""
    dev, counts, _ = _list_of(grads, "grads", _FLOATS)
    n = len(grads)
    table = _rows(_addresses(grads), counts, [_DT[t.dtype] for t in grads])
    nb = int(lib.gm_grad_norm_workspace_bytes(n))
    if out is None:
        buf = torch.empty(32 + nb // 8, dtype=torch.float64, device=dev)   # ws on 256 bytes
        out = GradNorm(buf.view(torch.float32)[2:3], buf[:1], buf.view(torch.int32)[3:4], buf[32:])
    else:
        _scalar(out.norm, torch.float32, "out.norm", dev)
        _scalar(out.scale, torch.float64, "out.scale", dev)
        _scalar(out.status, torch.int32, "out.status", dev)
        _ws_fits(out.ws, nb, "out.ws")
        if out.ws.device != dev:
            raise ValueError(f"out.ws: expected on {dev}, got {out.ws.device}")
    with _on(dev):
        _check(lib.gm_grad_norm(n, table, math.inf if max_norm is None else float(max_norm),
                                out.norm.data_ptr(), out.scale.data_ptr(), out.status.data_ptr(),
                                out.ws.data_ptr(), nb, _stream_of(dev)), "gm_grad_norm")
    return out


@dataclass
class AdamWState:
    """AdamW's moments of a list of parameters, on the device. ``bits`` 32: ``m``,
    ``v`` fp32; 8: uint8 codes with fp32 ``mscale``, ``vscale`` per 128 elements
    (the formats of gm_adamw_step). ``step``: completed steps, int64 [1]."""
    bits: int
    m: list
    v: list
    mscale: list
    vscale: list
    step: torch.Tensor
    scratch: torch.Tensor = field(default=None, repr=False)

    def __post_init__(self):
        if self.bits not in (32, 8):
            raise ValueError(f"bits: 32 or 8 expected, got {self.bits}")
        if self.scratch is None:
            self.scratch = torch.zeros(ADAMW_SCRATCH_BYTES, dtype=torch.uint8, device=self.step.device)

    @staticmethod
    def zeros(params, bits=32) -> "AdamWState":
        """The state before the first step of ``params`` (a list of tensors)."""
        if not params:
            raise ValueError("params: a non-empty list of tensors expected")
        dev = params[0].device
        numels = [p.numel() for p in params]

        def arena(dtype, per=1):   # one allocation, each tensor on a 256-element boundary
            at, spans = 0, []
            for n in numels:
                spans.append((at, -(-n // per)))
                at += -(-spans[-1][1] // 256) * 256
            flat = torch.zeros(at, dtype=dtype, device=dev)
            return [flat[a:a + n] for a, n in spans]
        if bits == 32:
            kept = [arena(torch.float32), arena(torch.float32), [], []]
        else:
            kept = [arena(torch.uint8), arena(torch.uint8), arena(torch.float32, GROUP),
                    arena(torch.float32, GROUP)]
        return AdamWState(bits, *kept, torch.zeros(1, dtype=torch.int64, device=dev))

    def tensors(self):
        return [*self.m, *self.v, *self.mscale, *self.vscale, self.step]

    def clone(self):
        c = lambda ts: [t.clone() for t in ts]                           # noqa: E731
        return AdamWState(self.bits, c(self.m), c(self.v), c(self.mscale), c(self.vscale),
                          self.step.clone())

    def check(self, numels, dev):
        """Raises ValueError unless the state fits tensors of `numels` elements."""
        kept = _F32 if self.bits == 32 else _U8
        _list_of(self.m, "m", kept, dev, numels)
        _list_of(self.v, "v", kept, dev, numels)
        if self.bits == 8:
            groups = [-(-n // GROUP) for n in numels]
            _list_of(self.mscale, "mscale", _F32, dev, groups)
            _list_of(self.vscale, "vscale", _F32, dev, groups)
        _scalar(self.step, torch.int64, "step", dev)
        if self.scratch.device != dev or not self.scratch.is_contiguous():
            raise ValueError(f"scratch: a contiguous tensor on {dev} expected")
        _ws_fits(self.scratch, ADAMW_SCRATCH_BYTES, "scratch")

    def moments(self, out=None):
        """(m, v) in fp32, two lists: the state's own tensors with 32-bit states, what
        the codes stand for with 8-bit ones (gm_adamw_unpack8; ``out``: two lists of
        fp32 tensors to write)."""
        if self.bits == 32:
            if out is not None:
                raise ValueError("out: 32-bit moments are the state's own tensors")
            return self.m, self.v
        numels = [t.numel() for t in self.m]
        dev = self.step.device
        self.check(numels, dev)
        if out is None:
            out = tuple([torch.empty(n, dtype=torch.float32, device=dev) for n in numels]
                        for _ in range(2))
        mo, vo = out
        _list_of(mo, "out[0]", _F32, dev, numels)
        _list_of(vo, "out[1]", _F32, dev, numels)
        table = _rows(*map(_addresses, (self.m, self.v, self.mscale, self.vscale, mo, vo)), numels)
        with _on(dev):
            _check(lib.gm_adamw_unpack8(len(numels), table, _stream_of(dev)),
                   "gm_adamw_unpack8")
        return mo, vo


class AdamWStep:
    """Marshals gm_adamw_step: ``step(state, params, grads)`` updates ``params`` and
    ``state`` in place, every tensor of the lists in one launch (one per combination
    of dtypes). params and grads: fp32, bf16 or fp16, each gradient of its
    parameter's size. eps: 1e-18 at least, with 8-bit states 1e-12."""

    def __init__(self, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, wd=0.01):
        self.lr, self.betas, self.eps, self.wd = float(lr), (float(betas[0]), float(betas[1])), \
            float(eps), float(wd)

    def __call__(self, state: AdamWState, params, grads, copies=None, clip: GradNorm | None = None,
                 skip=None, lr=None):
        """``copies``: 16-bit (or fp32) tensors that receive the new parameters rounded;
        ``clip``: a ``grad_norm`` result, whose factor scales the gradients and whose
        status makes the call change nothing; ``skip``: such a flag (int32 [1]) alone;
        ``lr``: this step's rate instead of the object's, a number or an fp32 [1]
        tensor on the device (read when the step runs, for captured graphs). A tensor that
        is written may overlap no other one of the lists (but ``copies[i]`` may be
        ``params[i]`` of the same dtype)."""
        dev, numels, pk = _list_of(params, "params", _FLOATS)
        _, _, gk = _list_of(grads, "grads", _FLOATS, dev, numels)
        state.check(numels, dev)
        ck = (torch.float32,)
        if copies is not None:
            _, _, ck = _list_of(copies, "copies", _FLOATS, dev, numels)
        if clip is not None:
            if skip is not None:
                raise ValueError("skip: clip brings its own flag")
            skip = clip.status
            _scalar(clip.scale, torch.float64, "clip.scale", dev)
        if skip is not None:
            _scalar(skip, torch.int32, "skip", dev)
        lr_dev = None
        if isinstance(lr, torch.Tensor):
            _scalar(lr, torch.float32, "lr", dev)
            lr_dev, lr = lr.data_ptr(), None
        n = len(numels)
        none = [0] * n
        columns = [_addresses(params), _addresses(grads), _addresses(state.m), _addresses(state.v),
                   _addresses(state.mscale) if state.bits == 8 else none,
                   _addresses(state.vscale) if state.bits == 8 else none,
                   _addresses(copies) if copies is not None else none, numels]
        prm = AdamWParams(self.lr if lr is None else float(lr), *self.betas, self.eps, self.wd,
                          state.bits, clip.scale.data_ptr() if clip is not None else None, lr_dev)
        flag = skip.data_ptr() if skip is not None else None
        table = _rows(*columns)
        with _on(dev):
            s = _stream_of(dev)
            if len(pk) == len(gk) == len(ck) == 1:
                status = lib.gm_adamw_step(n, table, *[_DT[next(iter(k))] for k in (pk, gk, ck)],
                                           ctypes.byref(prm), state.step.data_ptr(), flag,
                                           state.scratch.data_ptr(), s)
            else:
                kinds = [_DT[t.dtype] for ts in zip(params, grads, copies or params) for t in ts]
                status = lib.gm_adamw_step_mixed(n, table, struct.pack(f"{3 * n}i", *kinds), ctypes.byref(prm),
                                                 state.step.data_ptr(), flag, state.scratch.data_ptr(), s)
            if status != GM_OK:
                _repeated(columns, state.bits)
                _check(status, "gm_adamw_step")


def _repeated(columns, bits):
    """Names the list of a step that the library refused where a tensor is in it twice."""
    kept = [a for column in columns[2:6 if bits == 8 else 4] for a in column]
    for name, what in (("params", columns[0]), ("state", kept), ("copies", [a for a in columns[6] if a])):
        if len(set(what)) != len(what):
            raise ValueError(f"{name}: a tensor is in it more than once")


# ------------------------------------------------ microscaled 4-bit operands

MX4_BLOCK = {GM_MX4: 32, GM_NV4: 16}


def _mx4_padded(cols):
    return -(-cols // 128) * 128


@dataclass
class Mx4:
    """B matrices of ``rows`` x ``cols`` as microscaled 4-bit values along their rows
    (GM_MX4: blocks of 32, power-of-two scales; GM_NV4: blocks of 16, e4m3 scales and
    ``gscale`` [B]). With Kp = cols rounded up to 128: codes uint8 [B, rows, Kp / 2],
    scales uint8 [B, ceil(rows / 128), Kp / (4 block), 32, 4, 4]."""
    fmt: int
    rows: int
    cols: int
    codes: torch.Tensor
    scales: torch.Tensor
    gscale: torch.Tensor | None = None
    paired: bool = field(default=False, repr=False, compare=False)   # gscale is its transpose's too

    @staticmethod
    def empty(B, rows, cols, fmt, device=None, gscale=None):
        """An operand's buffers; ``gscale`` to share another operand's (its transpose's):
        the two are then one pair, to be written together."""
        if fmt not in MX4_BLOCK:
            raise ValueError(f"fmt: GM_MX4 or GM_NV4 expected, got {fmt}")
        dev = device or torch.device("cuda")
        kp = _mx4_padded(cols)
        paired = fmt == GM_NV4 and gscale is not None
        if fmt == GM_NV4 and gscale is None:
            gscale = torch.empty(B, dtype=torch.float32, device=dev)
        return Mx4(fmt, rows, cols,
                   torch.empty((B, rows, kp // 2), dtype=torch.uint8, device=dev),
                   torch.empty((B, -(-rows // 128), kp // (4 * MX4_BLOCK[fmt]), 32, 4, 4),
                               dtype=torch.uint8, device=dev), gscale, paired)

    def tensors(self):
        return [self.codes, self.scales] + ([self.gscale] if self.gscale is not None else [])

    def check(self, name="operand"):
        """Raises ValueError unless the tensors have the operand's layout; returns B."""
        c, s, g = self.codes, self.scales, self.gscale
        if self.fmt in MX4_BLOCK and self.rows >= 1 and self.cols >= 1 and c.dim() == 3:
            B, kp, dev = c.shape[0], _mx4_padded(self.cols), c.get_device()
            if (c.shape == (B, self.rows, kp // 2) and c.dtype == torch.uint8 and c.is_contiguous() and dev >= 0
                    and s.shape == (B, -(-self.rows // 128), kp // (4 * MX4_BLOCK[self.fmt]), 32, 4, 4)
                    and s.dtype == torch.uint8 and s.is_contiguous() and s.get_device() == dev
                    and (self.fmt == GM_MX4 or g is not None and g.shape == (B,) and g.dtype == torch.float32
                         and g.is_contiguous() and g.get_device() == dev)):
                return B
        self._error(name)

    def _error(self, name):
        """The first thing wrong with an operand that ``check`` refuses."""
        if self.fmt not in MX4_BLOCK:
            raise ValueError(f"{name}: fmt: GM_MX4 or GM_NV4 expected, got {self.fmt}")
        if self.rows < 1 or self.cols < 1 or self.codes.dim() != 3:
            raise ValueError(f"{name}: codes [B, rows, Kp / 2] of at least one row and column expected")
        B, kp = self.codes.shape[0], _mx4_padded(self.cols)
        parts = [("codes", self.codes, torch.uint8, (B, self.rows, kp // 2)),
                 ("scales", self.scales, torch.uint8,
                  (B, -(-self.rows // 128), kp // (4 * MX4_BLOCK[self.fmt]), 32, 4, 4))]
        if self.fmt == GM_NV4:
            if self.gscale is None:
                raise ValueError(f"{name}: gscale: expected shape {(B,)}")
            parts.append(("gscale", self.gscale, torch.float32, (B,)))
        for part, t, dt, shape in parts:
            if tuple(t.shape) != shape:
                raise ValueError(f"{name}: {part}: expected shape {shape}, got {tuple(t.shape)}")
            if t.dtype != dt:
                raise ValueError(f"{name}: {part}: dtype {t.dtype}, expected {dt}")
            if t.device != self.codes.device:
                raise ValueError(f"{name}: {part}: on {t.device}, expected on {self.codes.device}")
            if not t.is_contiguous():
                raise ValueError(f"{name}: {part}: expected a contiguous tensor")
        raise ValueError(f"{name}: expected a CUDA tensor")


def mx4_quant(X, fmt=GM_MX4, rows=True, cols=False, out=None):
    """Microscaled 4-bit operands of X [B, m, n] (or [m, n]; fp32, bf16 or fp16; rows of
    any stride, neighbouring elements of a row adjacent): of X itself (``rows``), of its
    transpose (``cols``, quantised along X's columns), or both from one pass, as a pair.
    The operands of a GM_NV4 pair share one ``gscale``. ``out``: the operand (or pair) to
    write into; an operand of a GM_NV4 pair is written together with the other one only,
    which would else stand for its old codes under the new matrix's scale."""
    B, m, n = _bmn(X)
    if X.dtype not in _DT:
        raise ValueError(f"X: dtype {X.dtype} is not one of {tuple(_DT)}")
    if fmt not in MX4_BLOCK:
        raise ValueError(f"fmt: GM_MX4 or GM_NV4 expected, got {fmt}")
    if not rows and not cols:
        raise ValueError("rows, cols: one of the two at least")
    if min(B, m, n) < 1:
        raise ValueError(f"X: empty ({tuple(X.shape)})")
    if not X.is_cuda:
        raise ValueError("X: expected a CUDA tensor")
    if n > 1 and X.stride(-1) != 1 or m > 1 and X.stride(-2) < n:
        raise ValueError(f"X: rows of adjacent elements that do not overlap expected, strides {X.stride()}")
    dev = X.device
    q = qt = None
    if out is not None:
        q, qt = out if rows and cols else (out, None) if rows else (None, out)
        for o, r, c, name in ((q, m, n, "out"), (qt, n, m, "out (columns)")):
            if o is None:
                continue
            if (o.fmt, o.rows, o.cols) != (fmt, r, c) or o.check(name) != B or o.codes.device != dev:
                raise ValueError(f"{name}: expected {B} operands of {r} x {c} in format {fmt} on {dev}")
        if q is not None and qt is not None:
            if fmt == GM_NV4 and q.gscale.data_ptr() != qt.gscale.data_ptr():
                raise ValueError("out: the two operands of one matrix share one gscale")
        elif (q or qt).paired:
            raise ValueError("out: one of a pair, whose other operand shares its gscale: write the pair, or an "
                             "operand of its own (Mx4.empty)")
    else:
        if rows:
            q = Mx4.empty(B, m, n, fmt, dev)
        if cols:
            qt = Mx4.empty(B, n, m, fmt, dev, gscale=q.gscale if rows else None)
    if rows and cols and fmt == GM_NV4:
        q.paired = qt.paired = True
    gs = (q or qt).gscale
    with _on(dev):
        _check(lib.gm_mx4_quant(B, m, n, X.data_ptr(), _DT[X.dtype], X.stride(-2) if m > 1 else n,
                                X.stride(0) if X.dim() == 3 and B > 1 else 0, fmt,
                                gs.data_ptr() if fmt == GM_NV4 else None,
                                q.codes.data_ptr() if rows else None, q.scales.data_ptr() if rows else None,
                                qt.codes.data_ptr() if cols else None,
                                qt.scales.data_ptr() if cols else None, _stream_of(dev)), "gm_mx4_quant")
    return (q, qt) if rows and cols else q if rows else qt


def mx4_dequant(q: Mx4, out=None, dtype=torch.float32):
    """What an operand stands for, [B, rows, cols] in ``dtype`` (gm_mx4_dequant)."""
    B = q.check("q")
    dev = q.codes.device
    if out is None:
        out = torch.empty((B, q.rows, q.cols), dtype=dtype, device=dev)
    _expect(out, (B, q.rows, q.cols), tuple(_DT), "out")
    if out.device != dev:
        raise ValueError(f"out: expected on {dev}, got {out.device}")
    with _on(dev):
        _check(lib.gm_mx4_dequant(B, q.rows, q.cols, q.fmt, q.codes.data_ptr(), q.scales.data_ptr(),
                                  q.gscale.data_ptr() if q.fmt == GM_NV4 else None, _ptr(out),
                                  _DT[out.dtype], _stream_of(dev)), "gm_mx4_dequant")
    return out


def mx4_matmul(A: Mx4, Bm: Mx4, out_dtype=torch.bfloat16, out=None, accumulate=False):
    """A Bm^T, [B, A.rows, Bm.rows], of two operands with the same columns and format;
    ``accumulate`` adds to ``out``. A linear layer's forward is mx4_matmul(X, W), its
    gradients mx4_matmul(dY, W's columns) and mx4_matmul(dY's columns, X's columns)."""
    B, B2 = A.check("A"), Bm.check("Bm")
    if (A.fmt, A.cols, B) != (Bm.fmt, Bm.cols, B2):
        raise ValueError(f"A and Bm: format, columns and batch differ: {(A.fmt, A.cols, B)} "
                         f"and {(Bm.fmt, Bm.cols, B2)}")
    dev = A.codes.device
    if Bm.codes.device != dev:
        raise ValueError(f"Bm: expected on {dev}, got {Bm.codes.device}")
    if out is None:
        if accumulate:
            raise ValueError("accumulate: needs out")
        out = torch.empty((B, A.rows, Bm.rows), dtype=out_dtype, device=dev)
    _expect(out, (B, A.rows, Bm.rows), tuple(_DT), "out")
    if out.device != dev:
        raise ValueError(f"out: expected on {dev}, got {out.device}")
    nv = A.fmt == GM_NV4
    with _on(dev):
        _check(lib.gm_mx4_matmul(B, A.rows, Bm.rows, A.cols, A.fmt, A.codes.data_ptr(),
                                 A.scales.data_ptr(), A.gscale.data_ptr() if nv else None,
                                 Bm.codes.data_ptr(), Bm.scales.data_ptr(),
                                 Bm.gscale.data_ptr() if nv else None, _ptr(out), _DT[out.dtype],
                                 int(bool(accumulate)), _stream_of(dev)), "gm_mx4_matmul")
    return out
