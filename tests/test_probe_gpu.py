"""The matrix-core probes: refusals, and rates below the datasheet's."""

from __future__ import annotations

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FP4_PEAK_TFLOPS = 256 * 4 * 4096 * 2.4e9 / 1e12


def _probe():
    return ctypes.CDLL(os.path.join(ROOT, "matrix_orthogonalizing_optimizer_amd", "libmoprobe.so"))


def test_fp4_probe_refuses():
    t = ctypes.c_double()
    f = _probe().mo_probe_mfma_fp4
    assert f(1, 0, 1, ctypes.byref(t)) == -2 and f(1, 1, 0, ctypes.byref(t)) == -2 and f(0, 1, 1, None) == -2


@pytest.mark.gpu
def test_fp4_probe_rates():
    t = ctypes.c_double()
    rates = []
    for random_codes in (0, 1):
        assert _probe().mo_probe_mfma_fp4(random_codes, 2000, 3, ctypes.byref(t)) == 0
        rates.append(t.value)
    # a loop of nothing else: at least a quarter of the peak even at the power limit's clock
    assert all(FP4_PEAK_TFLOPS / 4 < r < FP4_PEAK_TFLOPS * 1.05 for r in rates), rates
