"""The probe of the 8-bit matrix instruction: refusals, and rates below the datasheet's."""

from __future__ import annotations

import ctypes

import pytest

from test_probe_gpu import _probe

FP8_PEAK_TFLOPS = 256 * 4 * 2048 * 2.4e9 / 1e12


def test_fp8_probe_refuses():
    t = ctypes.c_double()
    f = _probe().mo_probe_mfma_fp8
    assert f(1, 0, 1, ctypes.byref(t)) == -2 and f(1, 1, 0, ctypes.byref(t)) == -2 and f(0, 1, 1, None) == -2
    assert f(3, 1, 1, ctypes.byref(t)) == -2 and f(-1, 1, 1, ctypes.byref(t)) == -2


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [0, 1, 2])
def test_fp8_probe_rates(codes):
    t = ctypes.c_double()
    assert _probe().mo_probe_mfma_fp8(codes, 2000, 3, ctypes.byref(t)) == 0
    # a loop of nothing else: at least a quarter of the peak even at the power limit's clock
    assert FP8_PEAK_TFLOPS / 4 < t.value < FP8_PEAK_TFLOPS * 1.05, t.value
