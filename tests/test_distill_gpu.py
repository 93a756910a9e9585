"""GPU parity of the token log probabilities and of the distillation loss with
its gradient against the fp64 oracle.

Tolerances count fp32 roundings (u = 2^-24).  With d = (x - m) / tau:
  * d itself: a subtraction, the rounded 1 / tau, a product: 3 u |d|;
  * e^d as a power of two: two more roundings of the argument and one step of
    the result: relative 5 u |d| + 2 u;
  * a sum over the row, each thread's part in order and a tree over parts
    (at least 256 of them, or whole vectors of them): V / 256 + 32 roundings;
  * log S: two steps of |log S| <= ln V.
The errors of d average over the row with weight e^d / S: sum p |d| <= ln V.
"""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from oracle import distill as od

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.float32, torch.bfloat16]


def _np(x):
    return x.detach().cpu().double().numpy()


def _sum_err(v):
    """Relative error of S."""
    lv = math.log(v) + 1.0
    return U * (v / 256 + 32 + 5 * lv + 2)


def _logits(rows, vocab, dtype, seed, pad=0, off=0, spread=4.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, vocab + pad + off, generator=g) * spread
    return z.to(dtype).cuda()[:, off:off + vocab]


def _close(got, want, tol):
    got, want = _np(got), np.asarray(want, np.float64)
    tol = np.broadcast_to(tol, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (got, want)
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    ok = ~np.isnan(want) & ~inf
    err = np.abs(got[ok] - want[ok])
    assert np.all(err <= tol[ok]), (float((err - tol[ok]).max()), got[ok][err > tol[ok]][:4], want[ok][err > tol[ok]][:4])


def _check_logprobs(z, tok, top, tau):
    rows, vocab = z.shape
    r = mo.token_logprobs(z, tok, top=top, temperature=tau)
    z64 = _np(z)
    lp, ent, tlp, tix = od.token_logprobs(z64, None if tok is None else _np(tok).astype(np.int64), top, tau)
    assert np.array_equal(r.top_index.cpu().numpy(), tix)
    lv = math.log(vocab) + 1.0
    fixed = _sum_err(vocab) + 4 * U * lv

    def tol_l(l):                             # |d| <= |l| + ln V
        a = np.nan_to_num(np.abs(l), posinf=0.0)
        return fixed + U * (3 * (a + lv) + a)

    _close(r.top_logprob, tlp, tol_l(tlp))
    if tok is None:
        assert r.logprob is None
    else:
        _close(r.logprob, lp, tol_l(lp))
    # entropy: log S and the mean of -d, whose terms are off by 5 u d^2 + ...
    with np.errstate(invalid="ignore", over="ignore"):
        zt = z64 / tau
        d = zt - zt.max(1, keepdims=True)
        p = np.exp(d)
        p = p / p.sum(1, keepdims=True)
        d1 = np.where(p > 0, p * -d, 0.0).sum(1)
        d2 = np.where(p > 0, p * d * d, 0.0).sum(1)
    tol = fixed + 5 * U * d2 + d1 * (2 * _sum_err(vocab) + 8 * U) + U * np.nan_to_num(np.abs(ent))
    _close(r.entropy, ent, np.nan_to_num(tol) + 1e-12)
    return r


VOCABS = [1, 2, 63, 255, 1000, 1023, 4096, 8193, 20001, 32000, 50001]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_logprobs(vocab, dtype):
    rows = 5
    z = _logits(rows, vocab, dtype, vocab)
    g = torch.Generator().manual_seed(vocab)
    tok = torch.randint(0, vocab, (rows,), generator=g)
    tok[1] = -1
    tok[2] = vocab                            # not a column
    for top in sorted({0, 1, min(5, vocab), min(64, vocab), min(128, vocab)}):
        _check_logprobs(z, tok.cuda(), top, 1.0)
    _check_logprobs(z, None, min(3, vocab), 0.3)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,pad,off", [(1001, 7, 0), (8190, 3, 1), (32000, 1, 5), (130001, 6, 3), (200003, 0, 0)])
def test_logprobs_strided_long_rows(vocab, pad, off, dtype):
    z = _logits(3, vocab, dtype, 3, pad, off)
    _check_logprobs(z, torch.tensor([0, vocab - 1, 17]).cuda(), 40, 2.0)
    _check_logprobs(z[1:2], torch.tensor([5]).cuda(), 7, 1.0)


@pytest.mark.parametrize("vocab", [300, 9000, 70000])
def test_logprobs_ties_take_the_lowest_columns(vocab):
    """All equal; two values; one column above a plateau; a descending and an
    ascending row; signed zeros."""
    z = torch.zeros(6, vocab)
    z[1, 1::2] = 1.0
    z[2, vocab // 2] = 3.0
    z[3] = -torch.arange(vocab) / 64.0
    z[4] = torch.arange(vocab) / 64.0
    z[5, ::2] = -0.0
    for dtype in DTYPES:
        _check_logprobs(z.to(dtype).cuda(), torch.arange(6).cuda(), 128, 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [77, 5000, 40000])
def test_logprobs_masked_and_special_rows(vocab, dtype):
    z = _logits(9, vocab, dtype, 5).clone()
    z[0] = -math.inf                          # nothing left
    z[1] = -math.inf
    z[1, vocab - 1] = 2.0                     # one token left
    z[2, : vocab - 9] = -math.inf             # fewer left than asked for
    z[3, 7] = math.nan
    z[4, 11] = math.inf
    z[5] = torch.finfo(dtype).min             # masked with the lowest value
    z[5, 3] = 0.0
    z[6] = torch.finfo(dtype).min
    z[7, 5], z[7, 9], z[7, 10] = math.nan, math.inf, math.nan
    z[8] = math.nan
    _check_logprobs(z, torch.tensor([0, vocab - 1, 3, 7, 11, 3, 3, 2, 0]).cuda(), 32, 1.0)


def test_logprobs_adversarial_order():
    """Every large value in columns that one thread of a strided walk would
    own, and many more equal values than slots."""
    z = torch.full((4, 65536), -5.0)
    z[0, ::1024] = torch.arange(64).float()
    z[1, ::512] = 4.0
    z[2, 32768:] = 1.0
    z[3, :8192] = torch.arange(8192).float() / 8192
    for dtype in DTYPES:
        _check_logprobs(z.to(dtype).cuda(), torch.tensor([0, 1, 2, 3]).cuda(), 128, 1.0)
        for row in range(4):
            _check_logprobs(z[row:row + 1].to(dtype).cuda(), torch.tensor([0]).cuda(), 100, 1.0)


def test_logprobs_many_rows():
    z = _logits(700, 333, torch.bfloat16, 8)
    _check_logprobs(z, (torch.arange(700) % 333).cuda(), 4, 1.0)


# ------------------------------------------------------------------ distillation
def _teacher(rows, vocab, k, seed):
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(vocab, generator=g)[:k] if vocab >= k else
                       torch.randint(0, vocab, (k,), generator=g) for _ in range(rows)])
    val = torch.randn(rows, k, generator=g) * 3
    return idx, val


def _check_distill(z, idx, val, tau, g=None, grad=True):
    rows, vocab = z.shape
    k = idx.shape[1]
    loss, dz = mo.distill_loss(z, idx.cuda(), val.cuda(), temperature=tau,
                               grad_loss=None if g is None else g.cuda(), grad=grad)
    z64 = _np(z)
    want, dwant = od.distill(z64, idx.numpy(), val.numpy(), tau, None if g is None else g.numpy())
    lv, lk = math.log(vocab) + 1.0, math.log(k) + 1.0
    tol = np.zeros(rows)
    gtol = np.zeros(dwant.shape)
    for r in range(rows):
        here = idx[r].numpy() >= 0
        i, t = idx[r].numpy()[here], val[r].numpy()[here].astype(np.float64) / tau
        if np.isnan(want[r]) or i.size == 0 or np.all(t == -np.inf):
            continue
        logp = od.log_softmax(t)
        p = np.exp(logp)
        logq = od.log_softmax(z64[r] / tau)
        # each log is off by 3 u |d| + (sum) + 4 u ln + u |l|; p by 5 u |d| + 2 u + (sum) + u
        el = np.where(p > 0, 4 * U * (np.abs(logp) + lk) + U * (k + 16 + 7 * lk), 0.0)
        eq = np.where(p > 0, 4 * U * (np.abs(logq[i]) + lv) + _sum_err(vocab) + 4 * U * lv, 0.0)
        ep = U * (5 * (np.abs(logp) + lk) + k + 24 + 5 * lk)
        pd = np.where(p > 0, p, 0.0)
        with np.errstate(invalid="ignore"):
            diff = np.where(p > 0, np.abs(logp - logq[i]), 0.0)
        tol[r] = tau * tau * np.nan_to_num(np.sum(pd * (el + eq) + np.nan_to_num(pd * ep) * diff + (k + 16) * U * pd * diff),
                                           posinf=0.0)
        if grad:
            gr = 1.0 if g is None else float(g[r])
            q = np.exp(logq)
            eqr = np.nan_to_num(U * 5 * (np.abs(logq) + lv), posinf=0.0) + _sum_err(vocab) + 8 * U
            et = q * eqr
            np.add.at(et, i, np.nan_to_num(pd * ep) + pd * U * (k + 4))
            gtol[r] = abs(gr) * tau * et * (1 + HALF[z.dtype]) + HALF[z.dtype] * np.abs(dwant[r]) + 2.0 ** -133
    _close(loss, want, tol + 1e-12)
    if grad:
        assert dz.dtype == z.dtype and dz.shape == z.shape
        _close(dz, dwant, gtol)
    else:
        assert dz is None
    return loss, dz


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_distill(vocab, dtype):
    rows = 6
    z = _logits(rows, vocab, dtype, vocab + 1)
    for k, tau in ((1, 1.0), (min(7, vocab), 2.0), (64, 0.5), (128, 1.0)):
        idx, val = _teacher(rows, vocab, k, vocab + k)
        idx[1] = -1                           # no teacher: skipped
        if k > 3:
            idx[2, 1:3] = -1                  # absent slots anywhere
            idx[3, 2] = idx[3, 0]             # a column named twice
            val[4, 1] = -math.inf
        g = torch.tensor([1.0, 1.0, 0.25, -2.0, 0.0, 1e-3])
        _check_distill(z, idx, val, tau, g)
        _check_distill(z, idx, val, tau, None, grad=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,pad,off", [(1001, 7, 0), (8190, 3, 1), (32000, 1, 5), (130001, 6, 3), (200003, 0, 0)])
def test_distill_strided_long_rows(vocab, pad, off, dtype):
    for rows in (1, 3):
        z = _logits(rows, vocab, dtype, 3, pad, off)
        idx, val = _teacher(rows, vocab, 20, 4)
        idx[0, 0], idx[0, 1] = 0, vocab - 1   # the row's ends
        loss, dz = _check_distill(z, idx, val, 1.0)
        # the same into a padded buffer, whose other columns stay
        buf = torch.full((rows, vocab + 9), 7.0, dtype=dtype, device="cuda")
        l2, g2 = mo.distill_loss(z, idx.cuda(), val.cuda(), out_grad=buf[:, 4:4 + vocab])
        assert torch.equal(g2, dz) and torch.equal(l2, loss)
        assert bool((buf[:, :4] == 7.0).all()) and bool((buf[:, 4 + vocab:] == 7.0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [77, 5000, 140000])
def test_distill_masked_and_special_rows(vocab, dtype):
    z = _logits(13, vocab, dtype, 6).clone()
    idx, val = _teacher(13, vocab, 5, 6)
    idx = idx % (vocab // 2)
    g = torch.ones(13)
    z[0] = -math.inf                          # student gives nothing: NaN
    z[1, vocab // 2:] = -math.inf             # masked columns without a teacher: finite
    z[2, idx[2, 3]] = -math.inf               # a teacher's token that the student excludes: +inf
    z[3, 7] = math.nan
    z[4, 11] = math.inf
    z[5] = math.nan
    idx[5] = -1                               # skipped whatever its logits
    z[6] = math.nan
    g[6] = 0.0                                # no gradient whatever its logits
    val[7] = -math.inf                        # no weight anywhere: skipped
    idx[8, 2] = vocab                         # not a column
    val[9, 1] = math.nan
    val[10, 4] = math.inf
    idx[11, 0], val[11, 0] = -1, math.nan     # an absent slot's logit is not read
    z[12] = torch.finfo(dtype).min
    z[12, 1] = 0.0
    _check_distill(z, idx, val, 1.0, g)
    for r in (0, 2, 5, 6, 8):                 # alone: as few rows as can be
        _check_distill(z[r:r + 1], idx[r:r + 1], val[r:r + 1], 1.0, g[r:r + 1])


def test_distill_gradient_against_differences():
    """Central differences of the GPU's own losses along a direction v: the
    step adds h^2 / 6 of a third derivative below 8 / tau (|v| <= 1), the
    losses' errors come in over h."""
    rows, vocab, h = 4, 500, 2.0 ** -5
    z = _logits(rows, vocab, torch.float32, 9, spread=2.0)
    idx, val = _teacher(rows, vocab, 9, 10)
    v = torch.randint(-1, 2, (rows, vocab), generator=torch.Generator().manual_seed(1)).float().cuda()
    for tau in (1.0, 2.0):
        _, dz = mo.distill_loss(z, idx.cuda(), val.cuda(), temperature=tau)
        up, _ = mo.distill_loss(z + h * v, idx.cuda(), val.cuda(), temperature=tau, grad=False)
        dn, _ = mo.distill_loss(z - h * v, idx.cuda(), val.cuda(), temperature=tau, grad=False)
        num = (_np(up) - _np(dn)) / (2 * h)
        tol = h * h / 6 * 8 / tau + tau * tau * (2 * _sum_err(vocab) + 40 * U * 20) / h + 4 * U * 10 / h
        assert np.all(np.abs((_np(dz) * _np(v)).sum(1) - num) <= tol)


def test_distill_many_rows_and_loss_alone():
    z = _logits(600, 333, torch.bfloat16, 8)
    idx, val = _teacher(600, 333, 4, 9)
    loss, _ = _check_distill(z, idx, val, 1.0)
    assert torch.equal(mo.distill_loss(z, idx.cuda(), val.cuda(), grad=False)[0], loss)


def test_empty_batches():
    z = torch.empty(0, 100, device="cuda")
    r = mo.token_logprobs(z, torch.empty(0, dtype=torch.int64, device="cuda"), top=3)
    assert r.logprob.shape == (0,) and r.top_index.shape == (0, 3)
    loss, g = mo.distill_loss(z, torch.empty(0, 2, dtype=torch.int64, device="cuda"), torch.empty(0, 2, device="cuda"))
    assert loss.shape == (0,) and g.shape == (0, 100)


def test_refusals_leave_outputs_alone():
    z = _logits(2, 100, torch.float32, 1)
    idx, val = _teacher(2, 100, 3, 1)
    out = torch.full((2, 100), 5.0, device="cuda")
    with pytest.raises(mo.MuonError):
        mo.distill_loss(z, idx.cuda(), val.cuda(), temperature=0.0, out_grad=out)
    with pytest.raises(mo.MuonError, match="overlap"):
        mo.distill_loss(z, idx.cuda(), val.cuda(), out_grad=z)
    assert bool((out == 5.0).all())
