"""GPU parity of the linear cross entropy against the fp64 oracle.

The operands are the bf16 values that the products take, so their products are
exact in fp32.  With S = max over v of sum_h |x_th w_vh|, a logit is off by d =
(H + 1) 2^-23 S at most.  Of the row's statistics, exponents of z log2(e) - m
are rounded once (2^-24 of at most |z - m| log2(e)) and the power of two itself
by 2^-22; V sums add V 2^-23 at most, in practice far less, and logs 2^-22 of
their value: the loss is off by 2 d + e, e = 2^-21 (2 + max|z| + |loss|) + min(V,
4096) 2^-23, and p relatively by as much, r = 2 (d + e).  dz = g (p - [target])
is then off by |g| (p r + 2^-22), rounded to bf16 (2^-8 of it) or to three terms
(2^-24), and the sums of the gradients add (n + 1) 2^-23 of their magnitudes, n
the length of the contraction, and half a step of the result.
"""

from __future__ import annotations

import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from oracle import linear_ce as oc

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def _inputs(t, h, v, seed, xd=BF16, wd=BF16, pad=0, skip=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(v, h + pad, generator=g, device="cuda") * (0.5 / h ** 0.5)
    x = torch.randn(t, h + pad, generator=g, device="cuda") * 2
    y = torch.randint(0, v, (t,), generator=g, device="cuda")
    x[:, :h] += w[y][:, :h] * (20 * torch.rand(t, 1, generator=g, device="cuda"))
    y = torch.where(torch.rand(t, generator=g, device="cuda") < skip, torch.full_like(y, -1), y)
    gl = torch.randn(t, generator=g, device="cuda")
    return x.to(xd)[:, :h], w.to(wd)[:, :h], y, gl


def _check(x, w, y, g, loss, dx, dw, add=None):
    o = oc.cross_entropy(x, w, y, g)
    v, h = w.shape
    xb, wb = x.bfloat16().double(), w.bfloat16().double()
    live = y >= 0
    xb = torch.where(live[:, None], xb, torch.zeros_like(xb))
    size = (xb.abs() @ wb.abs().t()).amax(1)
    d = (h + 1) * 2.0 ** -23 * size
    e = 2.0 ** -21 * (2 + o.logits.abs().amax(1) + o.loss.abs()) + min(v, 4096) * 2.0 ** -23
    assert loss.dtype == F32 and not bool(loss[~live].any())
    bad = (loss.double() - o.loss).abs() > 2 * d + e
    assert not bool(bad.any()), (loss[bad][:4], o.loss[bad][:4])
    if dx is None and dw is None:
        return
    ga = (torch.ones_like(o.loss) if g is None else g.double()).abs()[:, None]
    p = torch.softmax(o.logits, 1)
    ddz = torch.where(live[:, None], ga * (p * (2 * (d + e))[:, None] + 2.0 ** -22), torch.zeros_like(p))
    # what the gradients of one type take as dz is off by this besides
    for got, a, b, want, more in ((dx, o.dz, wb, o.dx, None), (dw, o.dz.t(), xb, o.dw, add)):
        if got is None:
            continue
        step = {BF16: 2.0 ** -8, F32: 2.0 ** -24}[got.dtype]
        off = (ddz if a is o.dz else ddz.t()) + step * a.abs() * 1.01
        tol = off @ b.abs() + (a.shape[1] + 1) * 2.0 ** -23 * (a.abs() @ b.abs())
        if more is not None:
            want = want + more.double()
            tol = tol + 2.0 ** -23 * more.double().abs()
        tol = tol + HALF[got.dtype] * 1.02 * want.abs() + 2.0 ** -133
        bad = (got.double() - want).abs() > tol
        assert not bool(bad.any()), (bad.nonzero()[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


SHAPES = [(1, 1, 1), (1, 64, 500), (3, 33, 100), (2, 8, 2), (64, 64, 257), (65, 130, 1000), (130, 257, 700), (300, 520, 1500),
          (7, 2048, 4099), (257, 100, 64), (1000, 65, 70), (513, 960, 3001)]
TYPES = [(BF16, BF16, BF16), (BF16, F32, F32), (F32, BF16, F32), (F32, F32, BF16)]


@pytest.mark.parametrize("t,h,v", SHAPES)
@pytest.mark.parametrize("xd,wd,dwd", TYPES)
def test_loss_and_gradients(t, h, v, xd, wd, dwd):
    x, w, y, g = _inputs(t, h, v, t + h + v, xd, wd)
    dw = torch.full((v, h), 7.0, dtype=dwd, device="cuda")
    loss, dx, got = mo.linear_cross_entropy(x, w, y, grad_loss=g, dw=dw)
    assert got is dw and dx.dtype == xd
    _check(x, w, y, g, loss, dx, dw)
    # the same bits again, and each part alone
    l2, dx2, dw2 = mo.linear_cross_entropy(x, w, y, grad_loss=g, dw=torch.empty_like(dw))
    assert torch.equal(loss, l2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    l3, none, none2 = mo.linear_cross_entropy(x, w, y, grad=False)
    assert none is None and none2 is None
    _check(x, w, y, None, l3, None, None)


@pytest.mark.parametrize("part", ["x", "weight"])
def test_one_gradient(part):
    x, w, y, g = _inputs(150, 200, 900, 3)
    loss, dx, dw = mo.linear_cross_entropy(x, w, y, grad_loss=g, grad=part)
    assert (dx is None) == (part == "weight") and (dw is None) == (part == "x")
    _check(x, w, y, g, loss, dx, dw)


@pytest.mark.parametrize("dwd", [F32, BF16])
def test_strided_operands_and_accumulation(dwd):
    """Rows apart, shifted starts; dw is added to, and what lies between its rows stays."""
    for pad, off in ((0, 0), (3, 1), (8, 8), (64, 0)):
        x, w, y, g = _inputs(70, 192 + off, 300, 5, pad=pad)
        x, w = x[:, off:], w[:, off:]
        buf = torch.randn(300, 192 + pad + off, device="cuda").to(dwd)
        keep, dw = buf.clone(), buf[:, off:off + 192]
        add = dw.clone()
        loss, dx, _ = mo.linear_cross_entropy(x, w, y, grad_loss=g, dw=dw, accumulate=True)
        _check(x, w, y, g, loss, dx, dw, add)
        keep[:, off:off + 192] = dw
        assert torch.equal(buf, keep)


@pytest.mark.parametrize("t,h,v,wd,dwd", [
    (2200, 64, 33000, BF16, BF16),        # logits computed twice, tiles of 256
    (2200, 72, 33000, F32, F32),          # the same, packed operands, three terms
    (9000, 64, 33000, BF16, BF16),        # the same in several pieces of dz
    (4500, 72, 33001, F32, F32),
    (4500, 256, 33001, BF16, F32),        # kept logits, several pieces of dz
    (50, 130, 1400001, F32, F32),         # weights copied for each product, logits computed twice
    (24, 20000, 27001, F32, BF16),        # the same with kept logits, several pieces of weights
    (40, 20000, 53000, BF16, F32),        # ones that are read in place
    (8192, 256, 131000, BF16, BF16),      # kept logits of 4.3 GB
    (40, 4096, 33000, BF16, F32),         # kept logits
    (24, 4100, 33000, F32, BF16),
    (4500, 128, 15001, BF16, BF16),       # computed twice, odd columns
    (3, 4, 4194300, F32, BF16),           # more rows of weights than 65535 times 64
])
def test_pieces(t, h, v, wd, dwd):
    x, w, y, g = _inputs(t, h, v, 11, BF16, wd)
    dw = torch.empty(v, h, dtype=dwd, device="cuda")
    loss, dx, _ = mo.linear_cross_entropy(x, w, y, grad_loss=g, dw=dw)
    _check(x, w, y, g, loss, dx, dw)
    # other pieces, whose statistics are joined in another order
    l2, dx2, _ = mo.linear_cross_entropy(x, w, y, grad_loss=g, dw=dw, grad="weight")
    assert dx2 is None
    _check(x, w, y, g, l2, None, dw)


@pytest.mark.parametrize("t,h,v", [(1, 64, 70000), (31, 200, 5003), (32, 129, 4097), (33, 1025, 9000), (64, 2048, 20011),
                                   (47, 68, 1027), (5, 1, 2049), (64, 130, 1024)])
@pytest.mark.parametrize("xd,wd", [(BF16, BF16), (F32, BF16), (BF16, F32)])
def test_dx_of_few_rows(t, h, v, xd, wd):
    """Weights read along their rows: odd sizes, several shares of the vocabulary,
    rows that end inside a block, and skipped rows that hold NaN."""
    x, w, y, g = _inputs(t, h, v, 3 * t + h, xd, wd)
    y[0] = v - 1
    loss, dx, dw = mo.linear_cross_entropy(x, w, y, grad_loss=g, grad="x")
    assert dw is None
    _check(x, w, y, g, loss, dx, None)
    bad = x.clone()
    bad[y < 0] = float("nan")
    l2, dx2, _ = mo.linear_cross_entropy(bad, w, y, grad_loss=g)
    assert torch.equal(loss, l2) and torch.equal(dx, dx2) and not bool(dx[y < 0].any())


def test_rows_that_take_no_part():
    """Skipped rows and rows with g = 0 may hold anything; all skipped; no rows."""
    x, w, y, g = _inputs(90, 100, 400, 7, skip=0.3)
    g = torch.where(torch.arange(90, device="cuda") % 4 == 1, torch.zeros_like(g), g)
    quiet = (y < 0) | (g == 0)
    bad = x.clone()
    bad[y < 0] = float("nan")
    bad[(y < 0) & (torch.arange(90, device="cuda") % 2 == 0)] = float("inf")
    loss, dx, dw = mo.linear_cross_entropy(bad, w, y, grad_loss=g)
    l2, dx2, dw2 = mo.linear_cross_entropy(x, w, y, grad_loss=g)
    assert torch.equal(loss, l2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    assert not bool(dx[quiet].any()) and not bool(loss[y < 0].any())
    _check(x, w, y, g, l2, dx2, dw2)
    # a row that is only scored: its loss follows its logits, its gradients do not
    bad = x.clone()
    bad[g == 0] = float("nan")
    loss, dx, dw = mo.linear_cross_entropy(bad, w, y, grad_loss=g)
    assert bool(loss[(g == 0) & (y >= 0)].isnan().all()) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    loss, dx, dw = mo.linear_cross_entropy(bad, w, torch.full_like(y, -1))
    assert not bool(loss.any()) and not bool(dx.any()) and not bool(dw.any())
    for dt in (BF16, F32):
        dw = torch.full((400, 100), 5.0, dtype=dt, device="cuda")
        loss, dx, _ = mo.linear_cross_entropy(x[:0], w, y[:0], dw=dw, accumulate=True)
        assert loss.shape == (0,) and dx.shape == (0, 100) and bool((dw == 5).all())
        mo.linear_cross_entropy(x[:0], w, y[:0], dw=dw)
        assert not bool(dw.any())


def test_targets_past_the_vocabulary_and_infinite_weights():
    x, w, y, g = _inputs(50, 64, 300, 9, skip=0.1)
    y[4] = 300
    y[5] = 1 << 40
    y[6] = 12
    loss, dx, dw = mo.linear_cross_entropy(x, w, y)
    hit = (torch.arange(50, device="cuda") == 4) | (torch.arange(50, device="cuda") == 5)
    assert bool(loss[hit].isnan().all()) and not bool(loss[~hit].isnan().any())
    assert bool(dx[hit].isnan().all()) and not bool(dx[~hit].isnan().any()) and bool(dw.isnan().all())
    y[4], y[5] = -1, -1
    w = w.clone()
    w[17, 3] = float("inf")                                     # logits of both infinities
    loss, dx, dw = mo.linear_cross_entropy(x, w, y)
    up = x[:, 3] > 0
    live = y >= 0
    assert bool(loss[up & live].isnan().all()) and not bool(loss[~live].any()) and not bool(dx[~live].any())
    down = (x[:, 3] < 0) & live & (y != 17)
    assert bool(torch.isfinite(loss[down]).all())               # -inf is a token of probability zero
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[17] = False
    rest = torch.where(y > 17, y - 1, y)
    l2 = mo.linear_cross_entropy(x, w[keep], rest, grad=False)[0]
    assert float((loss[down] - l2[down]).abs().max()) <= 2.0 ** -20


def test_large_logits_do_not_overflow():
    x, w, y, _ = _inputs(40, 64, 200, 13)
    x, w = x * 64, w * 64                                       # logits of tens of thousands
    loss, dx, dw = mo.linear_cross_entropy(x, w, y)
    _check(x, w, y, None, loss, dx, dw)
    assert bool(torch.isfinite(dw).all())


@pytest.mark.parametrize("scale", [1.0, 1e-30, 3e-39, 1e30])
def test_scale_of_the_gradient(scale):
    """dz is formed relative to the largest g: the gradients are that scale's times those of g = 1."""
    x, w, y, _ = _inputs(60, 64, 300, 15)
    one = mo.linear_cross_entropy(x.float(), w.float(), y)
    got = mo.linear_cross_entropy(x.float(), w.float(), y, grad_loss=torch.full((60,), scale, device="cuda"))
    g = float(torch.tensor(scale, dtype=F32))
    for a, b in zip(one[1:], got[1:]):
        assert float((a.double() * g - b.double()).abs().max()) <= 2.0 ** -23 * g * float(a.abs().max()) + 2.0 ** -149


def test_leading_axes():
    x, w, y, g = _inputs(24, 64, 100, 17)
    x = x.contiguous()
    flat = mo.linear_cross_entropy(x, w, y)
    loss, dx, dw = mo.linear_cross_entropy(x.view(2, 12, 64), w, y.view(2, 12))
    assert loss.shape == (24,) and dx.shape == (2, 12, 64)
    assert torch.equal(loss, flat[0]) and torch.equal(dx.view(24, 64), flat[1]) and torch.equal(dw, flat[2])
