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
