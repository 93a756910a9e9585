"""Checks of the 4-bit layer's arguments against each other: they come before
any work, so they run without a GPU."""

from __future__ import annotations

import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo

TOKENS, N, K = 5, 40, 64


def _image(rows, cols):
    return mo.Mx4Matrix.empty(rows, cols, "cpu")


def test_backward_refuses_images_of_different_layers():
    dy, x_t, w_t = torch.zeros(TOKENS, N), _image(K, TOKENS), _image(K, N)
    with pytest.raises(ValueError, match="features"):
        mo.mx4_linear_backward(dy, _image(K + 1, TOKENS), w_t)
    with pytest.raises(ValueError, match="features"):
        mo.mx4_linear_backward(dy, x_t, _image(K - 32, N))
    with pytest.raises(ValueError, match="GPU"):           # the right ones get as far as the device
        mo.mx4_linear_backward(dy, x_t, w_t)


@pytest.mark.parametrize("kw,word", [
    (dict(accumulate=True), "accumulate"),
    (dict(dw=torch.zeros(N, K + 1)), "dw must be"),
    (dict(dw=torch.zeros(N * K)), "dw must be"),
    (dict(dw=torch.zeros(K, N), accumulate=True), "dw must be"),
])
def test_backward_checks_dw_before_any_work(kw, word):
    with pytest.raises(ValueError, match=word):
        mo.mx4_linear_backward(torch.zeros(TOKENS, N), _image(K, TOKENS), _image(K, N), **kw)
