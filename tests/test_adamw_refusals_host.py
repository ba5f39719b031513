"""Settings that an AdamW step refuses, by the C entry point (never launched: no step count)."""

import ctypes

import numpy as np
import pytest

from bit_muon_optimizer_b200 import gmuon as gm


@pytest.mark.parametrize("bits,least", [(32, 1e-18), (8, 1e-12)])
def test_eps_below_the_least_is_refused(bits, least):
    table = np.array([[4096 * (1 + k) for k in range(6)] + [0, 8]], dtype=np.int64)
    for eps, b2 in ((least * 0.99, 0.999), (1e-30, 0.5), (0.0, 0.9), (least, 1 - 1e-14)):
        prm = gm.AdamWParams(1e-3, 0.9, b2, eps, 0.0, bits, None, None)
        assert gm.lib.gm_adamw_step(1, table.ctypes.data, 0, 0, 0, ctypes.byref(prm), None,
                                    None, 4096 * 10, None) == gm.GM_E_ARG, (eps, b2)
        assert b"eps" in gm.lib.gm_last_error()


def test_mixed_lists_are_checked_whole():
    """By the C entry point, without a step count (nothing can be launched)."""
    ok = [4096 * (1 + k) for k in range(6)]

    def call(rows, kinds, bits=32, count=None):
        table, kinds = np.array(rows, dtype=np.int64), np.array(kinds, dtype=np.int32)
        prm = gm.AdamWParams(1e-3, 0.9, 0.999, 1e-8, 0.0, bits, None, None)
        return (gm.lib.gm_adamw_step_mixed(len(rows) if count is None else count, table.ctypes.data, kinds.ctypes.data,
                                           ctypes.byref(prm), None, None, 4096 * 30, None),
                gm.lib.gm_last_error())
    far = lambda k, **kw: [kw.get(n, a + k * 65536) for n, a in zip(("p", "g", "m", "v", "ms", "vs"), ok)] \
        + [kw.get("copy", 0), kw.get("numel", 8)]                                   # noqa: E731
    good = [far(0), far(1)]
    for rows, kinds, what in [
            ([far(0), far(1, p=65536 + 4097)], [[0, 0, 0], [1, 0, 0]], b"tensor 1"),
            ([far(0), far(1, g=65536 + 4098)], [[0, 0, 0], [1, 0, 0]], b"tensor 1"),
            ([far(0), far(1, copy=65536 + 4097)], [[0, 0, 0], [0, 0, 1]], b"tensor 1"),
            ([far(0), far(1, numel=0)], [[0, 0, 0], [1, 0, 0]], b"tensor 1"),
            (good, [[0, 0, 0], [3, 0, 0]], b"dtype"), (good, [[0, 0, 0], [0, -1, 0]], b"dtype"),
            (good, [[0, 0, 0], [1, 0, 0]], b"NULL step")]:
        status, err = call(rows, kinds)
        assert status == gm.GM_E_ARG and what in err, (err, what)
    assert call([far(0), far(1, vs=0)], [[0, 0, 0], [1, 1, 1]], bits=8)[0] == gm.GM_E_ARG
    assert call(good, [[0, 0, 0]] * 2, count=0)[0] == call(good, [[0, 0, 0]] * 2, count=27 * 65536 + 1)[0] == gm.GM_E_ARG
    many = [far(k % 7) for k in range(65537)]
    status, err = call(many, [[1, 1, 1]] * len(many))
    assert status == gm.GM_E_ARG and b"65537" in err


def _row(k, **kw):
    """Arrays of 8 elements, 64 bytes apart, from address (k + 1) 65536 on."""
    at = [(k + 1) * 65536 + 64 * j for j in range(7)]
    return [kw.get(n, a) for n, a in zip(("p", "g", "m", "v", "ms", "vs", "copy"), at)] + [kw.get("numel", 8)]


OVERLAPS = [   # (what the second tensor has where), with the first at 65536
    dict(copy=65536),                                     # a copy that is another parameter
    dict(p=65536 + 64 * 6),                               # a parameter that is another's copy
    dict(copy=65536 + 64 * 2), dict(copy=65536 + 64 * 3), # a copy that is a state
    dict(p=65536 + 16), dict(m=65536 + 64 * 2 + 4),       # the middle of another array
    dict(m=65536 + 64 * 3 - 4),                           # its last element reaches into one
    dict(g=65536), dict(g=65536 + 64 * 6 + 28), dict(p=65536 + 64), # a gradient that is written
    dict(copy=2 * 65536 + 64 * 2), dict(g=2 * 65536), dict(v=2 * 65536 + 64 * 2),   # within one tensor
]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("order", [1, -1])
def test_overlapping_arrays_are_refused(bits, mixed, order):
    def call(*rows):
        rows = rows[::order]
        table = np.array(rows, dtype=np.int64)
        prm = gm.AdamWParams(1e-3, 0.9, 0.999, 1e-8, 0.0, bits, None, None)
        if mixed:
            kinds = np.zeros((len(rows), 3), dtype=np.int32)
            args = (len(rows), table.ctypes.data, kinds.ctypes.data, ctypes.byref(prm), None, None, 4096, None)
            return gm.lib.gm_adamw_step_mixed(*args), gm.lib.gm_last_error()
        args = (len(rows), table.ctypes.data, 0, 0, 0, ctypes.byref(prm), None, None, 4096, None)
        return gm.lib.gm_adamw_step(*args), gm.lib.gm_last_error()
    # what is in order gets as far as the missing step count
    for rows in ([_row(0), _row(1)], [_row(0), _row(1, g=65536 + 64)], [_row(0, copy=65536), _row(1, copy=0)],
                 [_row(0, numel=16), _row(1)], [_row(k) for k in range(100)]):
        status, err = call(*rows)
        assert status == gm.GM_E_ARG and b"NULL step" in err, err
    for kw in OVERLAPS:
        status, err = call(_row(0), _row(1, **kw))
        assert status == gm.GM_E_ARG and b"overlap" in err, (kw, err)
    status, err = call(_row(0, numel=17), _row(1))              # one element too long for its place
    assert status == gm.GM_E_ARG and b"overlap" in err
    if bits == 8:
        for kw in (dict(ms=65536 + 64 * 5), dict(vs=2 * 65536 + 64 * 2), dict(ms=2 * 65536 + 64 * 5)):
            status, err = call(_row(0), _row(1, **kw))
            assert status == gm.GM_E_ARG and b"overlap" in err, kw


def test_a_16_bit_copy_may_not_be_its_parameter():
    table = np.array([_row(0, copy=65536)], dtype=np.int64)
    prm = gm.AdamWParams(1e-3, 0.9, 0.999, 1e-8, 0.0, 32, None, None)
    for cdt, what in ((0, b"NULL step"), (1, b"overlap")):
        assert gm.lib.gm_adamw_step(1, table.ctypes.data, 0, 0, cdt, ctypes.byref(prm), None, None, 4096,
                                    None) == gm.GM_E_ARG and what in gm.lib.gm_last_error()


def test_overlapping_moments_are_refused():
    good = [65536 * (1 + j) for j in range(6)] + [100]
    for col, to in ((4, 5), (4, 0), (5, 1), (5, 2), (4, 3)):
        row = list(good)
        row[col] = good[to]
        table = np.array([row], dtype=np.int64)
        assert gm.lib.gm_adamw_unpack8(1, table.ctypes.data, None) == gm.GM_E_ARG
        assert b"overlap" in gm.lib.gm_last_error()
