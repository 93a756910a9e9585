"""Cross entropy of tokens that the model is certain of: what is left of their
loss and gradient, 1 - p, comes out to its own digits, not to those of 1.

Row t has a hidden column of its own, x = L_t there, and its target's weight is 1
there: its logits are L at the target and 0 elsewhere, 1 - p = (V - 1) / (e^L + V
- 1).  A term exp(-L) is off by (3 L + 4) 2^-24 of itself, a sum of V of them by
(V + 2) 2^-24, a quotient and log1p by 2^-22: r = (3 L + V + 16) 2^-24 in all, of
the loss, of 1 - p and of each p, as long as they are normal numbers.  Three bf16
terms hold dz to 2^-24; one to 2^-8, and a bf16 result is off by 2^-8 again.
"""

from __future__ import annotations

import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


@pytest.mark.parametrize("t,h,v", [(12, 12, 100), (60, 64, 1000), (60, 64, 5001), (150, 150, 4097),
                                   (2200, 64, 33000)])                      # the last one multiplies its logits again
@pytest.mark.parametrize("dt", [F32, BF16])
def test_what_is_left_of_a_certain_token(t, h, v, dt):
    n = min(t, h)                                                           # rows with a column of their own; the others are skipped
    gen = torch.Generator(device="cuda").manual_seed(t + v)
    at = torch.randperm(v, generator=gen, device="cuda")[:n]
    at[0], at[1] = v - 1, 0
    at = torch.where(torch.arange(n, device="cuda") > 1, at.clamp(1, v - 2), at)
    rows = torch.randperm(t, generator=gen, device="cuda")[:n]
    keep = torch.tensor([int(a) not in at[:i].tolist() for i, a in enumerate(at)], device="cuda")
    at, rows = at[keep], rows[keep]                                         # each target once
    n = len(at)
    lift = torch.arange(n, device="cuda") % 61                              # 0 to 60, exact in bf16
    col = torch.arange(n, device="cuda")
    x, w = torch.zeros(t, h, device="cuda"), torch.zeros(v, h, device="cuda")
    x[rows, col] = lift.float()
    w[at, col] = 1.0
    y = torch.full((t,), -1, dtype=torch.int64, device="cuda")
    y[rows] = at
    g = torch.randn(t, generator=gen, device="cuda")
    loss, dx, dw = mo.linear_cross_entropy(x.to(dt), w.to(dt), y, grad_loss=g)

    e = torch.exp(lift.double())
    left, p = (v - 1) / (e + v - 1), 1 / (e + v - 1)                        # 1 - p of the target, p of another column
    r = (3 * lift.double() + v + 16) * 2.0 ** -24
    want = torch.log1p((v - 1) * torch.exp(-lift.double()))
    assert bool(((loss[rows].double() - want).abs() <= r * want).all()), (loss[rows], want)
    gr = g[rows].double()
    # dx: column s of row t is dz of the target of s; dw: column t of a target's weights is dz times L
    dz = p[:, None].expand(n, n).clone()
    dz[col, col] = -left
    dz *= gr[:, None]
    tol = (r[:, None] + 2 * HALF[dt] + 2.0 ** -22) * dz.abs()
    for got, f in ((dx[rows][:, :n], torch.ones_like(lift)), (dw[at][:, :n].t(), lift)):
        bad = (got.double() - dz * f[:, None]).abs() > tol * f[:, None]
        assert not bool(bad.any()), (bad.nonzero()[:4], got[bad][:4], (dz * f[:, None])[bad][:4])


def test_one_column():
    """A vocabulary of one: the loss and both gradients are nothing."""
    x = torch.randn(70, 40, device="cuda")
    w = torch.randn(1, 40, device="cuda")
    loss, dx, dw = mo.linear_cross_entropy(x, w, torch.zeros(70, dtype=torch.int64, device="cuda"))
    assert not bool(loss.any()) and not bool(dx.any()) and not bool(dw.any())
