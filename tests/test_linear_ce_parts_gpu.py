"""Ways through the linear cross entropy that only large calls take: an fp32 x
whose logits are made in pieces or twice, gradients that go past the caches and
are added to, and the largest logits that are kept.  Tolerances are those of
the small sizes."""

from __future__ import annotations

import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from test_linear_ce_gpu import _check, _inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("t,h,v,wd,dwd", [
    (2200, 72, 33000, F32, F32),          # logits computed twice, three terms of both
    (2200, 64, 33000, BF16, BF16),        # three terms of one, one of the other
    (4500, 72, 33001, F32, F32),          # several pieces, a shorter last one
    (4500, 256, 33001, BF16, F32),        # kept logits, several pieces
    (24, 20000, 27001, F32, BF16),        # several pieces along the weights' rows
    (50, 130, 1400001, F32, F32),         # the same, computed twice
])
def test_pieces_of_an_fp32_x(t, h, v, wd, dwd):
    x, w, y, g = _inputs(t, h, v, 21, F32, wd)
    dw = torch.empty(v, h, dtype=dwd, device="cuda")
    loss, dx, _ = mo.linear_cross_entropy(x, w, y, grad_loss=g, dw=dw)
    assert dx.dtype == F32
    _check(x, w, y, g, loss, dx, dw)
    l2, dx2, none = mo.linear_cross_entropy(x, w, y, grad_loss=g, grad="x")          # other pieces
    assert none is None
    _check(x, w, y, g, l2, dx2, None)


@pytest.mark.parametrize("t,h,v,dwd", [(100, 2048, 4200, F32), (100, 2048, 8300, BF16), (1100, 1024, 9000, F32)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradients_past_the_caches(t, h, v, dwd, accumulate):
    """dw of more than 32 MiB in whole lines, written and added to."""
    x, w, y, g = _inputs(t, h, v, 23)
    dw = torch.randn(v, h, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").to(dwd)
    assert dw.numel() * dw.element_size() > 32 << 20 and dw.data_ptr() % 128 == 0
    add = dw.clone() if accumulate else None
    loss, dx, _ = mo.linear_cross_entropy(x, w, y, grad_loss=g, dw=dw, accumulate=accumulate)
    _check(x, w, y, g, loss, dx, dw, add)


def test_the_largest_logits_that_are_kept():
    """4 GiB of them, to the last byte: the last row's target is the last column."""
    x, w, y, g = _inputs(8192, 256, 131072, 25)
    y[-1], y[-2], y[0] = 131071, 131070, 131071
    loss, dx, dw = mo.linear_cross_entropy(x, w, y, grad_loss=g)
    _check(x, w, y, g, loss, dx, dw)
    # its loss alone, from no kept logits
    one = mo.linear_cross_entropy(x[-1:], w, y[-1:], grad=False)[0]
    _check(x[-1:], w, y[-1:], None, one, None, None)
