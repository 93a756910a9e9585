"""GPU parity of the MX4 images and products against the fp64 oracle.

Images and the values read back are exact, so they must match bit for bit.
A product's terms are exact in fp32; K of them summed in fp32 in any order
are off by at most K 2^-23 sum |a b| (two half steps a term leave room for
the matrix cores' own alignment of a step's terms), and the result is rounded
once: half a step of its type, 2^-24 (fp32) or 2^-8 (bf16), relative.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from oracle import mx4 as om

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.float32, torch.bfloat16]
SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (1, 2048), (33, 1), (7, 64), (31, 96), (32, 32), (65, 130), (64, 256),
          (129, 257), (300, 100), (2, 4097), (515, 8)]


def _rand(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    x = x * torch.exp2(torch.randint(-8, 9, shape, generator=g).float())
    return x.to(dtype)


def _np(x):
    return x.detach().float().cpu().double().numpy()


def _same_image(q, x64):
    codes, scales = om.image(x64)
    assert q.shape == x64.shape
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)


def _same_values(t, want):
    got = _np(t)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_images_and_values(shape, dtype):
    x = _rand(shape, shape[0] * 1000 + shape[1], dtype)
    q, qt = mo.mx4_quantize(x.cuda(), images="both")
    x64 = _np(x)
    _same_image(q, x64)
    _same_image(qt, x64.T.copy())
    one, two = mo.mx4_quantize(x.cuda()), mo.mx4_quantize(x.cuda(), images="cols")
    assert torch.equal(one.codes, q.codes) and torch.equal(one.scales, q.scales)
    assert torch.equal(two.codes, qt.codes) and torch.equal(two.scales, qt.scales)
    for dt in DTYPES:
        _same_values(mo.mx4_dequantize(q, dtype=dt), om.rounded(x64))
        _same_values(mo.mx4_dequantize(qt, dtype=dt), om.rounded(x64.T))


def _edge_matrix():
    """Rows of special blocks: halfway cases at several scales, values next to
    a power of two, zeros of both signs, subnormals, the largest numbers, NaN
    and infinities."""
    rows = []
    half = [0.0, -0.0, 0.25, -0.25, 0.75, 1.25, 1.75, 2.5, -2.5, 3.5, 5.0, -5.0, 6.0, 7.0, 4.0, 0.125]
    for e in (0, -20, 40, -124, 120):
        rows.append([v * 2.0 ** e for v in half] * 2)
    for top in (4.0, 4.0 * (1 + 2.0 ** -7), 8.0 * (1 - 2.0 ** -8), 2.0 ** -126, 2.0 ** -125, 2.0 ** -124):
        rows.append([top, -top / 3, top / 7] + [top * i / 64 for i in range(29)])
    rows.append([0.0] * 32)
    rows.append([-0.0] * 32)
    rows.append([2.0 ** -133 * i for i in range(32)])
    rows.append([(-1) ** i * 2.0 ** -130 * i for i in range(32)])
    rows.append([3.3e38, -3.3e38] + [1e38] * 30)
    rows.append([float("nan")] + [1.0] * 31)
    rows.append([1.0] * 31 + [float("inf")])
    rows.append([-float("inf")] + [0.0] * 31)
    return torch.tensor(rows)


@pytest.mark.parametrize("dtype", DTYPES)
def test_special_blocks(dtype):
    x = _edge_matrix().to(dtype)
    x64 = x.double().numpy()           # keeps subnormals
    q = mo.mx4_quantize(x.cuda())
    _same_image(q, x64)
    qt = mo.mx4_quantize(x.t().contiguous().cuda(), images="cols")
    _same_image(qt, x64)
    for dt in DTYPES:
        got = mo.mx4_dequantize(q, dtype=dt).cpu().double().numpy()
        want = om.rounded(x64)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_and_shifted_sources(dtype):
    buf = _rand((70, 150), 3, dtype).cuda()
    for r0, r1, c0, c1 in [(0, 70, 0, 149), (1, 66, 1, 34), (3, 40, 7, 135), (0, 1, 5, 6), (5, 70, 8, 136)]:
        x = buf[r0:r1, c0:c1]
        q, qt = mo.mx4_quantize(x, images="both")
        _same_image(q, _np(x))
        _same_image(qt, _np(x).T.copy())


def test_list_of_many_matrices_and_out():
    """More matrices than one launch takes; images of an earlier call reused."""
    shapes = [(1 + 13 * i % 90, 1 + 29 * i % 170) for i in range(101)]
    xs = [_rand(s, i, torch.float32).cuda() for i, s in enumerate(shapes)]
    qs = mo.mx4_quantize(xs, images="both")
    for x, (q, qt) in zip(xs, qs):
        _same_image(q, _np(x))
        _same_image(qt, _np(x).T.copy())
    ys = [x * 3.0 for x in xs]
    again = mo.mx4_quantize(ys, images="both", out=qs)
    assert all(a[0] is b[0] and a[1] is b[1] for a, b in zip(again, qs))
    for y, (q, qt) in zip(ys, qs):
        _same_image(q, _np(y))
    for v, y in zip(mo.mx4_dequantize([q for q, _ in qs], dtype=torch.float32), ys):
        _same_values(v, om.rounded(_np(y)))


def test_padding_is_written():
    """Codes and scales behind the last column are zero whatever was there."""
    x = _rand((5, 37), 9, torch.bfloat16).cuda()
    q, qt = mo.Mx4Matrix.empty(5, 37, "cuda"), mo.Mx4Matrix.empty(37, 5, "cuda")
    for i in (q, qt):
        i.codes.fill_(255)
        i.scales.fill_(255)
    mo.mx4_quantize(x, images="both", out=(q, qt))
    _same_image(q, _np(x))
    _same_image(qt, _np(x).T.copy())


# ------------------------------------------------------------------- products
def _check_product(got, av, bv, k, add=None):
    want = av @ bv.T + (0.0 if add is None else add)
    size = np.abs(av) @ np.abs(bv).T + (0.0 if add is None else np.abs(add))
    g = got.detach().cpu().double().numpy()
    # the last rounding, of a value that is itself off by the sum's error
    tol = (k + 1) * 2.0 ** -23 * size + HALF[got.dtype] * np.abs(want) * (1 + 2.0 ** -6) + 2.0 ** -133
    assert np.array_equal(np.isnan(g), np.isnan(want))
    bad = np.nan_to_num(np.abs(g - want)) > np.nan_to_num(tol)
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], want[bad][:4])


MM = [(1, 1, 1), (1, 17, 33), (3, 5, 31), (16, 16, 128), (17, 33, 129), (1, 300, 2048), (2, 130, 4097), (15, 257, 500),
      (31, 64, 96), (64, 64, 512), (65, 63, 640), (128, 128, 1024), (129, 255, 1025), (200, 72, 3), (256, 256, 512),
      (257, 130, 2050), (300, 520, 64), (512, 384, 1536), (1, 2048, 64), (48, 1408, 70), (33, 1000, 5000),
      # several groups of stages, with whole and partial last ones, in tiles of every size
      (70, 100, 4130), (130, 90, 6176), (1500, 1700, 2111), (3900, 3301, 4300), (3900, 3301, 416)]


@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", MM)
def test_product(m, n, k, out_dtype):
    a, b = _rand((m, k), m + k, torch.float32).cuda(), _rand((n, k), 7 * n + k, torch.bfloat16).cuda()
    qa, qb = mo.mx4_quantize(a), mo.mx4_quantize(b)
    av, bv = _np(mo.mx4_dequantize(qa, dtype=torch.float32)), _np(mo.mx4_dequantize(qb, dtype=torch.float32))
    got = mo.mx4_matmul(qa, qb, out_dtype=out_dtype)
    _check_product(got, av, bv, k)
    assert torch.equal(got, mo.mx4_matmul(qa, qb, out_dtype=out_dtype))


@pytest.mark.parametrize("m,n,k", [(1, 40, 100), (20, 50, 300), (130, 257, 513), (256, 512, 1024)])
@pytest.mark.parametrize("out_dtype", DTYPES)
def test_accumulate_into_strided_rows(m, n, k, out_dtype):
    """Adds to out; the columns between the rows stay as they were."""
    a, b = mo.mx4_quantize(_rand((m, k), 1, torch.float32).cuda()), mo.mx4_quantize(_rand((n, k), 2, torch.float32).cuda())
    av, bv = _np(mo.mx4_dequantize(a, dtype=torch.float32)), _np(mo.mx4_dequantize(b, dtype=torch.float32))
    for pad, off in ((0, 0), (3, 1), (8, 8)):
        buf = _rand((m, n + pad + off), 3, out_dtype, 50.0).cuda()
        keep = buf.clone()
        out = buf[:, off:off + n]
        add = _np(out)
        assert mo.mx4_matmul(a, b, out=out, accumulate=True) is out
        _check_product(out, av, bv, k, add)
        keep[:, off:off + n] = out
        assert torch.equal(buf, keep)


def test_wide_scale_range_and_nan_blocks():
    """Block scales 2^-60 .. 2^60 across K, and a NaN block in one row."""
    g = torch.Generator().manual_seed(5)
    a = torch.randn(40, 700, generator=g) * torch.exp2(torch.linspace(-60, 60, 700))
    b = torch.randn(70, 700, generator=g) * torch.exp2(torch.linspace(50, -70, 700))
    a[7, 650] = float("nan")
    b[69, 3] = float("inf")
    qa, qb = mo.mx4_quantize(a.cuda()), mo.mx4_quantize(b.cuda())
    av, bv = om.rounded(a.double().numpy()), om.rounded(b.double().numpy())
    got = mo.mx4_matmul(qa, qb, out_dtype=torch.float32)
    assert torch.isnan(got[7]).all() and torch.isnan(got[:, 69]).all()
    _check_product(got, av, bv, 700)


def test_product_of_many_rows():
    """More row tiles than a grid's second axis has places."""
    m = 16 * 65536 + 5
    a = torch.zeros(m, 32, device="cuda")
    a[:, 0] = torch.arange(m, device="cuda") % 7 - 3.0
    b = torch.ones(1, 32, device="cuda")
    q = mo.mx4_quantize(a)
    got = mo.mx4_matmul(q, mo.mx4_quantize(b), out_dtype=torch.float32)
    assert torch.equal(got[:, 0], mo.mx4_dequantize(q, dtype=torch.float32)[:, 0])


# --------------------------------------------------------------------- linear
@pytest.mark.parametrize("t,n,k", [(1, 64, 96), (5, 33, 70), (130, 96, 257)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_and_backward(t, n, k, dtype):
    x, w = _rand((t, k), 1, dtype), _rand((n, k), 2, torch.float32, 0.05)
    dy = _rand((t, n), 3, dtype, 0.01)
    wq, wq_t = mo.mx4_quantize(w.cuda(), images="both")
    y, x_t = mo.mx4_linear(x.cuda(), wq, out_dtype=torch.float32, save=True)
    _check_product(y, om.rounded(_np(x)), om.rounded(_np(w)), k)
    dx, dw = mo.mx4_linear_backward(dy.cuda(), x_t, wq_t, dx_dtype=torch.float32)
    _check_product(dx, om.rounded(_np(dy)), om.rounded(_np(w).T), n)
    _check_product(dw, om.rounded(_np(dy).T), om.rounded(_np(x).T), t)
    # two micro-batches into one gradient
    both = dw.clone()
    mo.mx4_linear_backward(dy.cuda(), x_t, wq_t, dw=both, accumulate=True)
    _check_product(both, om.rounded(_np(dy).T), om.rounded(_np(x).T), t, add=_np(dw))


def test_linear_keeps_leading_axes_and_empty_batches():
    w = mo.mx4_quantize(_rand((40, 64), 1, torch.float32).cuda())
    x = _rand((6, 64), 2, torch.bfloat16).cuda()
    y = mo.mx4_linear(x, w)
    assert torch.equal(mo.mx4_linear(x.view(2, 3, 64), w), y.view(2, 3, 40))
    assert mo.mx4_linear(x[:0], w).shape == (0, 40)
    assert mo.mx4_linear(x.view(2, 3, 64)[:0], w).shape == (0, 3, 40)


def test_refusals_leave_outputs_alone():
    x = _rand((40, 64), 1, torch.float32).cuda()
    q = mo.mx4_quantize(x)
    with pytest.raises(ValueError, match="expected an image"):
        mo.mx4_quantize(x, out=mo.Mx4Matrix.empty(40, 65, "cuda"))
    out = torch.full((40, 39), 2.0, device="cuda")
    with pytest.raises(ValueError, match="out must be"):
        mo.mx4_matmul(q, q, out=out)
    # an image whose codes lie inside the output
    big = torch.zeros(40 * 40 * 2, dtype=torch.uint8, device="cuda")
    inside = mo.Mx4Matrix(big[:q.codes.numel()].view(q.codes.shape), q.scales, 64)
    with pytest.raises(mo.MuonError, match="overlaps"):
        mo.mx4_matmul(inside, q, out=big.view(torch.bfloat16).view(40, 40))
    assert not bool(big.any())
    assert bool((out == 2.0).all())
    before = (q.codes.clone(), q.scales.clone())
    with pytest.raises(mo.MuonError, match="columns"):
        mo.mx4_matmul(q, mo.mx4_quantize(_rand((3, 65), 1, torch.float32).cuda()))
    assert torch.equal(before[0], q.codes) and torch.equal(before[1], q.scales)
