"""The distillation loss and gradient over the whole range of temperatures,
from 2^-126 to 2^63, against the fp64 oracle (tolerances: test_distill_gpu)."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from oracle import distill as od
from test_distill_gpu import DTYPES, HALF, U, _logits, _np, _sum_err, _teacher

pytestmark = pytest.mark.gpu

TAUS = [2.0 ** -126, 1e-37, 1e-30, 2.0 ** -76, 1e-19, 1e-5, 0.125, 1.0, 64.0, 2.0 ** 20, 2.0 ** 62, 2.0 ** 63]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [500, 40001, 180001])
@pytest.mark.parametrize("tau", TAUS)
def test_loss_and_gradient_over_the_range(tau, vocab, dtype):
    """Errors relative to each row's own terms, with no absolute allowance
    beyond the subnormals' steps.  tau log p = (t - m) - tau ln s is off by
    half a step of the difference and of the product, s by k + 16 + 7 (ln k +
    1) roundings, and half a step of the result; tau log q alike with the
    row's sum; p by the exponent's five roundings of |d|, s and the quotient."""
    rows, k = 5, 6
    tau = float(np.float32(tau))
    z = _logits(rows, vocab, dtype, 17, spread=8.0).clone()
    idx, val = _teacher(rows, vocab, k, 18)
    z[0, int(idx[0, 2])] = 100.0              # the teacher's best is the student's: nearly no loss at small tau
    val[0, 2] = 50.0
    z[1, int(idx[1, 0])] = -40.0              # and far below it
    val[1, 0] = 60.0
    idx[2, 1] = idx[2, 4]                     # a column named twice
    z[3, 7] = torch.finfo(dtype).min          # masked columns without a teacher
    z[3, 8] = -math.inf
    idx[3] = torch.tensor([9, 10, 11, 12, 13, -1])
    g = torch.tensor([1.0, 0.5, -2.0, 1.0, 1.0])
    loss, dz = mo.distill_loss(z, idx.cuda(), val.cuda(), temperature=tau, grad_loss=g.cuda())
    z64 = _np(z)
    want, dwant = od.distill(z64, idx.numpy(), val.numpy(), tau, g.numpy())
    lv, lk = math.log(vocab) + 1.0, math.log(k) + 1.0
    got, dgot = _np(loss), _np(dz)
    with np.errstate(over="ignore"):
        held = want.astype(np.float32)        # what fp32 can hold: beyond it the loss is inf
    assert np.array_equal(np.isinf(got), np.isinf(held)), (got, want)
    for r in range(rows):
        here = idx[r].numpy() >= 0
        i, t = idx[r].numpy()[here], val[r].numpy()[here].astype(np.float64) / tau
        logp, logq = od.log_softmax(t), od.log_softmax(z64[r] / tau)
        p, q = np.exp(logp), np.exp(logq)
        p = np.where(p < 2.0 ** -126, 0.0, p)  # the exponential's flushed results
        pos = p > 0
        diff = np.where(pos, np.abs(logp - logq[i]), 0.0)
        el = np.where(pos, 4 * U * (np.abs(logp) + lk) + U * (k + 16 + 7 * lk), 0.0)
        eq = np.where(pos, 4 * U * (np.abs(logq[i]) + lv) + _sum_err(vocab) + 4 * U * lv, 0.0)
        ep = np.where(pos, U * (5 * (np.abs(logp) + lk) + k + 24 + 5 * lk), 0.0)
        flushed = np.sum(np.where(pos, 0.0, 2.0 ** -126 * np.abs(np.nan_to_num(logq[i]))))
        tol = tau * (tau * np.sum(p * (el + eq) + p * ep * diff + (k + 16) * U * p * diff) + tau * flushed) + 2.0 ** -148
        if not np.isinf(held[r]):
            assert abs(got[r] - want[r]) <= tol, (r, got[r], want[r], tol)
        live = q > 0
        et = np.where(live, q * (U * 5 * np.where(live, np.abs(logq) + lv, 0.0) + _sum_err(vocab) + 8 * U), 0.0) + 2.0 ** -126
        np.add.at(et, i, p * ep + p * U * (k + 4) + 2.0 ** -126)
        gtol = abs(float(g[r])) * tau * et * (1 + HALF[dtype]) + HALF[dtype] * np.abs(dwant[r]) + 2.0 ** -133
        err = np.abs(dgot[r] - dwant[r])
        assert np.all(err <= gtol), (r, float((err - gtol).max()))
