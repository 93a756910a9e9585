"""The linear cross entropy over the whole range of finite logits.

Only one hidden column is not zero, x in it is +-s and w a whole number up to
100: a logit is one product, exact in fp32 up to 100 s < 2^127.  A term exp(z -
max) is then off, relatively, by the rounding of the difference and of its
product with log2(e) (3 |z - max| 2^-24; terms past exp(-90) are nothing beside
the others' 2^-126) and the power of two (2^-22); V of them add (V + 2) 2^-24: p
by r = (3 * 90 + V + 8) 2^-24 of itself.  dz is off by |g| (p r + 2^-126) and, in
the target's column, by |g| 2^-22 more, its three terms by 2^-24 of it, and the
gradients' sums of n terms by (n + 1) 2^-23 of their magnitudes.  The loss, a
difference of logits and a logarithm: 2^-22 of itself and (V + 8) 2^-23.
"""

from __future__ import annotations

import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from oracle import linear_ce as oc

pytestmark = pytest.mark.gpu


def _one_column(t, h, v, s, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros(t, h, device="cuda")
    x[:, 0] = s * (torch.randint(0, 2, (t,), generator=g, device="cuda") * 2 - 1)
    w = torch.zeros(v, h, device="cuda")
    w[:, 0] = torch.randint(-100, 101, (v,), generator=g, device="cuda").float()
    y = torch.randint(0, v, (t,), generator=g, device="cuda")
    z = x[:, :1].double() @ w[:, :1].double().t()
    best = torch.arange(t, device="cuda") % 3 == 0                          # rows whose target is the likeliest
    y = torch.where(best, z.argmax(1), y)
    y[1] = -1
    return x, w, y, torch.randn(t, generator=g, device="cuda")


def _check(x, w, y, g, loss, dx, dw):
    o = oc.cross_entropy(x, w, y, g)
    t, v = o.dz.shape
    assert bool(((loss.double() - o.loss).abs() <= 2.0 ** -22 * o.loss.abs() + (v + 8) * 2.0 ** -23).all())
    ga = torch.where(y >= 0, g.double().abs(), torch.zeros_like(o.loss))[:, None]
    off = ga * (torch.softmax(o.logits, 1) * ((3 * 90 + v + 8) * 2.0 ** -24) + 2.0 ** -126) + 2.0 ** -24 * o.dz.abs()
    off[torch.arange(t, device="cuda"), y.clamp(min=0)] += 2.0 ** -22 * ga[:, 0]
    for got, want, a, e, b in ((dx, o.dx, o.dz, off, w.double()), (dw, o.dw, o.dz.t(), off.t(), x.double())):
        tol = (e + (a.shape[1] + 1) * 2.0 ** -23 * a.abs()) @ b.abs() + 2.0 ** -24 * want.abs() + 2.0 ** -126
        bad = (got.double() - want).abs() > tol                             # not of a NaN
        assert bool(torch.isfinite(got).all()) and not bool(bad.any()), (bad.nonzero()[:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("s", [1.0, 2.0 ** 24, 2.0 ** 31, 2.0 ** 40, 2.0 ** 100, 2.0 ** 120])
@pytest.mark.parametrize("t,h,v", [(40, 64, 300), (130, 65, 700),           # dx along the weights' rows, and as a product
                                   (2200, 64, 33000)])                      # logits multiplied again
def test_every_finite_logit(t, h, v, s):
    x, w, y, g = _one_column(t, h, v, s, 7)
    loss, dx, dw = mo.linear_cross_entropy(x, w, y, grad_loss=g)
    _check(x, w, y, g, loss, dx, dw)
    assert torch.equal(mo.linear_cross_entropy(x, w, y, grad=False)[0], loss)


def test_logits_whose_difference_passes_the_largest_number():
    """2^127 and -2^127: the difference is no fp32 number, the softmax is one-hot."""
    x = torch.full((3, 8), 0.0, device="cuda")
    x[:, 0] = 2.0 ** 100
    w = torch.zeros(5, 8, device="cuda")
    w[:, 0] = torch.tensor([1.0, -1.0, 0.0, -1.0, -1.0], device="cuda") * 2.0 ** 27
    y = torch.tensor([0, 2, 1], device="cuda")
    loss, dx, dw = mo.linear_cross_entropy(x, w, y)
    assert loss[:2].tolist() == [0.0, 2.0 ** 127] and bool(loss[2] > 3e38)   # 2^128, past the type
    assert dx[:, 0].tolist() == [0.0, 2.0 ** 27, 2.0 ** 28] and not bool(dx[:, 1:].any())
    assert dw[:, 0].tolist() == [2.0 ** 101, -2.0 ** 100, -2.0 ** 100, 0.0, 0.0]
