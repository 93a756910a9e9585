"""GPU parity of the router's balance loss against the fp64 oracle.

A probability is off by 2^-24 (6 + 1.5 (max - z)) relative at most: the exponent is
rounded twice and the power of two by 2^-22 in all, the sum and its reciprocal
by E 2^-24 or so; r = (E + 16 + 2 max|z - max|) 2^-23 covers it.  Means over n
tokens add n 2^-24 at most relative to their size (terms are of one sign), f is
off by 2^-23, and the gradient w / n p (f - sum f p) by (2 r + 2^-21) of w / n p (f
+ sum f p), plus half a step of its type.
"""

from __future__ import annotations

import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from oracle import linear_ce as oc

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def _inputs(t, e, k, seed, dtype, pad=0, drop=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = (torch.randn(t, e + pad, generator=g, device="cuda") * 2).to(dtype)[:, :e]
    idx = torch.topk(z.float() + 0.1 * torch.randn(t, e, generator=g, device="cuda"), min(k, e), dim=1)[1]
    if k > e:
        idx = torch.cat((idx, idx[:, :1].expand(t, k - e)), 1)
    idx = torch.where(torch.rand(t, 1, generator=g, device="cuda") < drop, torch.full_like(idx, -1), idx)
    idx = torch.where(torch.rand(t, k, generator=g, device="cuda") < drop, torch.full_like(idx, -7), idx)
    return z, idx.contiguous()


def _check(z, idx, got, weight, g, add=None):
    loss, counts, grad = oc.balance(z, idx, weight, g)
    t, e = z.shape
    live = (idx >= 0).any(1)
    zz = torch.where(live[:, None], z.double(), torch.zeros_like(z, dtype=torch.float64))
    r = (e + 16 + 2 * float((zz.amax(1, keepdim=True) - zz).amax()) if t else 0.0) * 2.0 ** -23
    assert torch.equal(got.counts, counts) and got.counts.dtype == torch.int64
    assert got.loss.shape == () and abs(float(got.loss) - float(loss)) <= (r + (t + 64) * 2.0 ** -23) * abs(float(loss))
    if got.grad is None:
        return
    f = counts.double() * e / max(1, int(counts.sum()))
    p = torch.where(live[:, None], torch.softmax(z.double(), 1), torch.zeros_like(zz))
    size = abs(weight * g) / max(1, int(live.sum())) * p * (f + (p * f).sum(1, keepdim=True))
    want = grad if add is None else grad + add.double()
    tol = (2 * r + 2.0 ** -21) * size + HALF[z.dtype] * 1.01 * want.abs() + 2.0 ** -133
    bad = (got.grad.double() - want).abs() > tol
    assert not bool(bad.any()), (bad.nonzero()[:4], got.grad[bad][:4], want[bad][:4])


SHAPES = [(0, 8, 2), (1, 1, 1), (1, 64, 6), (5, 3, 3), (37, 64, 6), (63, 17, 1), (256, 16, 2), (257, 64, 8), (1000, 33, 4), (5000, 64, 6),
          (40, 100, 8), (700, 128, 2), (300, 200, 20), (2049, 256, 8), (90, 500, 3), (3000, 512, 8), (33, 600, 70), (130, 1024, 4), (50, 4096, 9),
          (70000, 8, 2)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("t,e,k", SHAPES)
def test_loss_counts_and_gradient(t, e, k, dtype):
    z, idx = _inputs(t, e, k, t + e + k, dtype, pad=t % 3)
    g = torch.tensor(0.75, device="cuda")
    got = mo.balance_loss(z, idx, weight=0.02, grad_loss=g)
    _check(z, idx, got, 0.02, 0.75)
    again = mo.balance_loss(z, idx, weight=0.02, grad_loss=g)
    assert torch.equal(got.loss, again.loss) and torch.equal(got.grad, again.grad)
    alone = mo.balance_loss(z, idx, grad=False)
    assert alone.grad is None
    _check(z, idx, alone, 1.0, 1.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("t", [37, 3000])
def test_accumulates_into_strided_rows(t, dtype):
    z, idx = _inputs(t, 60, 4, 1, dtype, pad=5)
    buf = (torch.randn(t, 67, device="cuda") * 1e-3).to(dtype)
    keep, out = buf.clone(), buf[:, 3:63]
    add = out.clone()
    got = mo.balance_loss(z, idx, weight=5.0, out_grad=out, accumulate=True)
    assert got.grad is out
    _check(z, idx, got, 5.0, 1.0, add)
    keep[:, 3:63] = out
    assert torch.equal(buf, keep)
    mo.balance_loss(z, idx, weight=5.0, out_grad=out)
    _check(z, idx, mo.BalanceLoss(got.loss, got.counts, out), 5.0, 1.0)


@pytest.mark.parametrize("t", [20, 3000])
def test_tokens_without_a_choice_may_hold_anything(t):
    z, idx = _inputs(t, 48, 4, 2, F32)
    dead = (idx < 0).all(1)
    dead[3] = True
    idx[3] = -1
    clean = mo.balance_loss(z, idx)
    z2 = z.clone()
    z2[dead] = float("nan")
    z2[3] = float("inf")
    got = mo.balance_loss(z2, idx)
    assert torch.equal(got.loss, clean.loss) and torch.equal(got.grad, clean.grad) and not bool(got.grad[dead].any())
    none = mo.balance_loss(z2, torch.full_like(idx, -1))
    assert float(none.loss) == 0 and not bool(none.counts.any()) and not bool(none.grad.any())


@pytest.mark.parametrize("t", [20, 3000])
def test_masked_experts_and_bad_values(t):
    z, idx = _inputs(t, 48, 4, 3, F32, drop=0.0)
    z[:, 40:] = -float("inf")                                   # experts that are switched off
    idx = torch.topk(z, 4, dim=1)[1].contiguous()
    got = mo.balance_loss(z, idx)
    assert not bool(got.counts[40:].any()) and not bool(got.grad[:, 40:].any()) and bool(torch.isfinite(got.loss))
    z3 = z[:, :40].contiguous()
    less = mo.balance_loss(z3, idx)
    # f scales with the number of experts
    assert abs(float(got.loss) / float(less.loss) - 48 / 40) <= 2.0 ** -18
    z[7, 0] = float("nan")
    z[9] = -float("inf")
    got = mo.balance_loss(z, idx)
    rows = got.grad.isnan().any(1)
    assert bool(got.loss.isnan()) and bool(rows[7]) and bool(rows[9]) and int(rows.sum()) == 2
    z[7, 0], z[9] = 0.0, 0.0
    idx[2, 1] = 48
    got = mo.balance_loss(z, idx)
    assert bool(got.loss.isnan()) and bool(got.grad.isnan().any(1).all()) and int(got.counts.sum()) == 4 * t - 1


def test_an_expert_named_twice_counts_twice():
    z = torch.zeros(2, 4, device="cuda")
    got = mo.balance_loss(z, torch.tensor([[1, 1], [1, 3]], device="cuda"))
    assert got.counts.tolist() == [0, 3, 0, 1] and float(got.loss) == 1.0
