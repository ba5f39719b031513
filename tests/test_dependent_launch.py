"""Kernels that start before the kernel they depend on has ended read what that one
writes, so none of their pointers may be promised read-only for the kernel's life:
such a promise (const with __restrict__) lets a load be made through the cache that is
not coherent, or before the wait. Read from the sources, without a GPU."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_muon_optimizer_b200", "csrc")
WAIT = ("griddepcontrol.wait", "wait_for_previous()")


def _kernels(text):
    """(name, parameters, body) of every __global__ function."""
    for m in re.finditer(r"__global__\s+void\s*(?:__launch_bounds__\([^)]*\)\s*)?(\w+)\s*\(", text):
        at, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        params = text[m.end():at - 1]
        if text[at:].lstrip()[0] != "{":
            continue
        start = text.index("{", at)
        end, depth = start + 1, 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        yield m.group(1), params, text[start:end]


def test_the_reader_finds_the_kernels():
    found = {}
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        with open(path) as f:
            found.update({name: body for name, _, body in _kernels(f.read())})
    waiting = {n for n, body in found.items() if any(w in body for w in WAIT)}
    assert {"k_adamw", "k_grad_norm_join", "k_mx4_rows", "k_mx4_tile", "k_mx4_gemm"} <= waiting
    assert "k_adamw_begin" in found and "k_adamw_begin" not in waiting


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu"))), ids=os.path.basename)
def test_waiting_kernels_make_no_read_only_promise(path):
    with open(path) as f:
        for name, params, body in _kernels(f.read()):
            if any(w in body for w in WAIT):
                assert "__restrict__" not in params, f"{name}({params})"
                assert "__ldg(" not in body and "ld.global.nc" not in body, name
