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
