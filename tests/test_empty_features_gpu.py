"""Leading axes in front of an axis without features."""

from __future__ import annotations

import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from matrix_orthogonalizing_optimizer_amd import _flat2


@pytest.mark.parametrize("shape,flat", [((2, 3, 0), (6, 0)), ((2, 0, 0), (0, 0)), ((0,), (1, 0)), ((2, 3, 5), (6, 5)), ((2, 0, 5), (0, 5)),
                                        ((5,), (1, 5)), ((6, 0), (6, 0))])
def test_rows_of_leading_axes(shape, flat):
    assert _flat2(torch.empty(shape)).shape == flat


def test_cross_entropy_refuses_no_features():
    with pytest.raises(mo.MuonError, match="hidden"):
        mo.linear_cross_entropy(torch.empty(2, 3, 0), torch.empty(7, 0), torch.zeros(2, 3, dtype=torch.int64))


@pytest.mark.gpu
def test_a_layer_without_inputs_or_outputs():
    """The product of nothing is zeros, in x's shape."""
    w, w_t = mo.fp8_quantize(torch.empty(7, 0, device="cuda"), images="both")
    y, x_t = mo.fp8_linear(torch.empty(2, 3, 0, device="cuda"), w, save=True)
    assert y.shape == (2, 3, 7) and not bool(y.any()) and x_t.shape == (0, 6)
    dx, dw = mo.fp8_linear_backward(torch.ones(2, 3, 7, device="cuda"), x_t, w_t)
    assert dx.shape == (2, 3, 0) and dw.shape == (7, 0)
    w, w_t = mo.fp8_quantize(torch.empty(0, 5, device="cuda"), images="both")
    y, x_t = mo.fp8_linear(torch.ones(2, 3, 5, device="cuda"), w, save=True)
    assert y.shape == (2, 3, 0) and x_t.shape == (5, 6)
    dx, dw = mo.fp8_linear_backward(torch.empty(2, 3, 0, device="cuda"), x_t, w_t)
    assert dx.shape == (2, 3, 5) and not bool(dx.any()) and dw.shape == (0, 5)
