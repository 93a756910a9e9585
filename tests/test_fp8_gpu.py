"""GPU parity of the 8-bit images and products against the fp64 oracle.

Images and the values read back are exact, so they must match bit for bit.
A product with an fp32 output has exact terms; K of them summed in fp32 in any
order are off by at most K 2^-23 sum |a b| (two half steps a term leave room
for the matrix cores' own alignment of a step's terms), and the result is
rounded once: 2^-24 relative.  For a bf16 output the instruction takes the
codes themselves and aligns groups of at most 16 products to the largest,
keeping 15 bits below it or more: each of a group's products is off by at most
2^-15 of the largest, which is at most the group's sum of magnitudes: 2^-11 sum
|a b| in all, beside the 2^-8 of the rounding.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from oracle import fp8 as of

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.float32, torch.bfloat16]
SHAPES = [(1, 1), (1, 127), (1, 128), (1, 129), (1, 2048), (129, 1), (7, 64), (127, 130), (128, 128), (129, 257), (256, 384),
          (300, 100), (2, 4097), (515, 8), (64, 2065)]


def _rand(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    x = x * torch.exp2(torch.randint(-16, 3, shape, generator=g).float())
    return x.to(dtype)


def _np(x):
    return x.detach().float().cpu().double().numpy()


def _same_image(q, x64, square=False):
    codes, scales = of.image(x64, square)
    assert q.shape == x64.shape
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)


def _same_values(t, want):
    got = t.detach().cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_images_and_values(shape, dtype, square):
    x = _rand(shape, shape[0] * 1000 + shape[1], dtype)
    q, qt = mo.fp8_quantize(x.cuda(), images="both", square=square)
    x64 = _np(x)
    _same_image(q, x64, square)
    _same_image(qt, x64.T.copy(), square)
    one, two = mo.fp8_quantize(x.cuda(), square=square), mo.fp8_quantize(x.cuda(), images="cols", square=square)
    assert torch.equal(one.codes, q.codes) and torch.equal(one.scales, q.scales)
    assert torch.equal(two.codes, qt.codes) and torch.equal(two.scales, qt.scales)
    for dt in DTYPES:
        _same_values(mo.fp8_dequantize(q, dtype=dt), of.rounded(x64, square))
        _same_values(mo.fp8_dequantize(qt, dtype=dt), of.rounded(x64.T.copy(), square))


def _edge_matrix():
    """Blocks of special values: halfway cases, largest values next to a scale's
    border, zeros of both signs, subnormals, the largest numbers, NaN, infinity."""
    rows = []
    for e in (0, -30, 40, -118, 119):
        rows.append([(1 + i / 16.0) * 2.0 ** (e - 7 + i % 15) * (-1) ** i for i in range(120)])   # every other one halfway
        rows.append([448.0 * 2.0 ** (e - 1)] + [i * 2.0 ** (e - 11) for i in range(119)])         # subnormal steps and halves
    for top in (448.0, 448.0 * (1 + 2.0 ** -23), 448.0 * (1 + 2.0 ** -7), 1.75, 1.75 * (1 + 2.0 ** -7), 2.0 ** -126, 448 * 2.0 ** -127,
                450 * 2.0 ** -127, 2.0 ** -133):
        rows.append([top, -top / 3, top / 7] + [top * i / 117 for i in range(117)])
    rows.append([0.0] * 120)
    rows.append([-0.0] * 120)
    rows.append([2.0 ** -133 * i for i in range(120)])
    rows.append([3.4028234e38, -3.4028234e38, 3.38e38, 3.25e38, 1e38] + [2.0 ** 100] * 115)
    rows.append([float("nan")] + [1.0] * 119)
    rows.append([1.0] * 119 + [float("inf")])
    rows.append([-float("inf")] + [0.0] * 119)
    return torch.tensor(rows, dtype=torch.float64).float()


@pytest.mark.parametrize("dtype", DTYPES)
def test_special_blocks(dtype):
    x = _edge_matrix().to(dtype)
    if dtype == torch.bfloat16:
        x = torch.where(x.isinf() & (x != _edge_matrix()), torch.full_like(x, 3.3895e38), x)      # rounded past bf16
    x64 = x.double().numpy()
    q = mo.fp8_quantize(x.cuda())
    _same_image(q, x64)
    qt = mo.fp8_quantize(x.t().contiguous().cuda(), images="cols")
    _same_image(qt, x64)
    _same_values(mo.fp8_dequantize(q, dtype=torch.float32), of.rounded(x64))
    # bf16 holds them all but the steps below its own, 2^-133
    got, want = mo.fp8_dequantize(q).cpu().double().numpy(), of.rounded(x64)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.max(np.abs(np.nan_to_num(got) - np.nan_to_num(want))) <= 2.0 ** -134


def test_every_code_reads_back():
    codes = torch.arange(256, dtype=torch.uint8).repeat(1, 1).cuda()
    for byte in (0, 1, 100, 127, 140, 246, 254, 255):
        scales = torch.zeros(1, 16, dtype=torch.uint8)
        scales[0, :2] = byte
        q = mo.Fp8Matrix(codes, scales.cuda(), 256)
        want = of.values(codes.cpu().numpy(), scales.numpy(), 256)
        got = mo.fp8_dequantize(q, dtype=torch.float32).cpu().double().numpy()
        with np.errstate(over="ignore"):
            want = want.astype(np.float32).astype(np.float64)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


def test_every_bf16_value():
    """All finite bf16 numbers, alone and below a power of two up to ten binades above them."""
    bits = torch.arange(0x7f80, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).float()
    for up in (0, 1, 7, 10):
        top = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -126))) + up).clamp(max=2.0 ** 127)
        m = torch.zeros(x.numel(), 3)
        m[:, 0], m[:, 1], m[:, 2] = x, -x, top if up else 0.0
        _same_image(mo.fp8_quantize(m.to(torch.bfloat16).cuda()), m.to(torch.bfloat16).double().numpy())


@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_and_shifted_sources(dtype, square):
    buf = _rand((170, 350), 3, dtype).cuda()
    for r0, r1, c0, c1 in [(0, 170, 0, 349), (1, 66, 1, 134), (3, 140, 7, 264), (0, 1, 5, 6), (5, 170, 8, 136)]:
        x = buf[r0:r1, c0:c1]
        q, qt = mo.fp8_quantize(x, images="both", square=square)
        _same_image(q, _np(x), square)
        _same_image(qt, _np(x).T.copy(), square)
        _same_image(mo.fp8_quantize(x, square=square), _np(x), square)


def test_list_of_many_matrices_and_out():
    """More matrices than one launch takes, some without elements; images of an earlier call reused."""
    shapes = [(1 + 13 * i % 190, 29 * i % 370) for i in range(101)]
    xs = [_rand(s, i, torch.float32).cuda() for i, s in enumerate(shapes)]
    qs = mo.fp8_quantize(xs, images="both")
    for x, (q, qt) in zip(xs, qs):
        _same_image(q, _np(x))
        _same_image(qt, _np(x).T.copy())
    ys = [x * 3.0 for x in xs]
    again = mo.fp8_quantize(ys, images="both", out=qs)
    assert all(a[0] is b[0] and a[1] is b[1] for a, b in zip(again, qs))
    for v, y in zip(mo.fp8_dequantize([q for q, _ in qs], dtype=torch.float32), ys):
        _same_values(v, of.rounded(_np(y)))
    rows = mo.fp8_quantize(xs)
    assert all(torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales) for a, b in zip(rows, mo.fp8_quantize(xs)))
    for x, q in zip(xs, rows):
        _same_image(q, _np(x))


def test_padding_is_written():
    x = _rand((5, 137), 9, torch.bfloat16).cuda()
    for square in (False, True):
        q, qt = mo.Fp8Matrix.empty(5, 137, "cuda"), mo.Fp8Matrix.empty(137, 5, "cuda")
        one = mo.Fp8Matrix.empty(5, 137, "cuda")
        for i in (q, qt, one):
            i.codes.fill_(255)
            i.scales.fill_(255)
        mo.fp8_quantize(x, images="both", square=square, out=(q, qt))
        mo.fp8_quantize(x, square=square, out=one)
        for i in (q, one):
            _same_image(i, _np(x), square)
        _same_image(qt, _np(x).T.copy(), square)


# ------------------------------------------------------------------- products
def _check_product(got, av, bv, k, add=None):
    a, b = torch.from_numpy(np.array(av)).cuda(), torch.from_numpy(np.array(bv)).cuda()
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    loose = 2.0 ** -11 * size if got.dtype == torch.bfloat16 else 0.0
    if add is not None:
        want, size = want + torch.from_numpy(add).cuda(), size + torch.from_numpy(np.abs(add)).cuda()
    g = got.double()
    # the last rounding, of a value that is itself off by the sum's error
    tol = (k + 1) * 2.0 ** -23 * size + loose + HALF[got.dtype] * want.abs() * (1 + 2.0 ** -6) + 2.0 ** -133
    assert torch.equal(g.isnan(), want.isnan())
    bad = (g - want).abs() > tol
    assert not bool(bad.any()), (bad.nonzero()[:4], g[bad][:4], want[bad][:4])


MM = [(1, 1, 1), (1, 17, 33), (3, 5, 127), (16, 16, 128), (17, 33, 129), (1, 300, 2048), (2, 130, 4097), (15, 257, 500),
      (31, 64, 96), (32, 700, 3000), (64, 64, 512), (65, 63, 640), (128, 128, 1024), (129, 255, 1025), (200, 72, 3), (256, 256, 512),
      (257, 130, 2050), (300, 520, 64), (512, 384, 1536), (1, 2048, 64), (48, 1408, 70), (33, 1000, 5000),
      # several groups of scales, with whole and partial last ones, in tiles of every size
      (70, 100, 4130), (130, 90, 6176), (1500, 1700, 2111), (2500, 3001, 4300), (3900, 3301, 416), (3900, 4100, 130)]


@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", MM)
def test_product(m, n, k, out_dtype):
    a, b = _rand((m, k), m + k, torch.float32).cuda(), _rand((n, k), 7 * n + k, torch.bfloat16).cuda()
    qa, qb = mo.fp8_quantize(a), mo.fp8_quantize(b)
    av, bv = _np(mo.fp8_dequantize(qa, dtype=torch.float32)), _np(mo.fp8_dequantize(qb, dtype=torch.float32))
    got = mo.fp8_matmul(qa, qb, out_dtype=out_dtype)
    _check_product(got, av, bv, k)
    assert torch.equal(got, mo.fp8_matmul(qa, qb, out_dtype=out_dtype))


@pytest.mark.parametrize("m,n,k", [(1, 40, 100), (20, 50, 300), (130, 257, 513), (256, 512, 1024), (1000, 900, 400)])
@pytest.mark.parametrize("out_dtype", DTYPES)
def test_accumulate_into_strided_rows(m, n, k, out_dtype):
    """Adds to out; the columns between the rows stay as they were."""
    a, b = mo.fp8_quantize(_rand((m, k), 1, torch.float32).cuda()), mo.fp8_quantize(_rand((n, k), 2, torch.float32).cuda())
    av, bv = _np(mo.fp8_dequantize(a, dtype=torch.float32)), _np(mo.fp8_dequantize(b, dtype=torch.float32))
    for pad, off in ((0, 0), (3, 1), (8, 8)):
        buf = _rand((m, n + pad + off), 3, out_dtype, 50.0).cuda()
        keep = buf.clone()
        out = buf[:, off:off + n]
        add = _np(out)
        assert mo.fp8_matmul(a, b, out=out, accumulate=True) is out
        _check_product(out, av, bv, k, add)
        keep[:, off:off + n] = out
        assert torch.equal(buf, keep)


@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("m,n", [(40, 70), (3, 70), (300, 260), (2100, 2050)])
def test_wide_scale_range_and_nan_blocks(m, n, out_dtype):
    """Block scales 2^-60 .. 2^60 across K, and NaN blocks in both operands, in tiles of every size."""
    g = torch.Generator().manual_seed(5)
    k = 1500
    a = torch.randn(m, k, generator=g) * torch.exp2(torch.linspace(-60, 60, k))
    b = torch.randn(n, k, generator=g) * torch.exp2(torch.linspace(50, -70, k))
    a[2, 1450] = float("nan")
    b[69, 3] = float("inf")
    qa, qb = mo.fp8_quantize(a.cuda()), mo.fp8_quantize(b.cuda())
    got = mo.fp8_matmul(qa, qb, out_dtype=out_dtype)
    assert bool(got[2].isnan().all()) and bool(got[:, 69].isnan().all())
    av, bv = mo.fp8_dequantize(qa, dtype=torch.float32), mo.fp8_dequantize(qb, dtype=torch.float32)
    _check_product(got, _np(av), _np(bv), k)


def test_extreme_scales():
    """Blocks whose values or whose other operand's lie at the ends of fp32: the products are ordinary numbers."""
    a = torch.full((4, 128), 2.0 ** -120)
    a[1] = 2.0 ** 127
    a[2] = 2.0 ** -100
    a[3, ::2] = 2.0 ** -128
    b = torch.full((3, 128), 2.0 ** 110)
    b[1] = 2.0 ** -110
    b[2] = 1.0
    for dt in DTYPES:
        got = mo.fp8_matmul(mo.fp8_quantize(a.cuda()), mo.fp8_quantize(b.cuda()), out_dtype=dt).double().cpu()
        want = a.double() @ b.double().t()
        want = torch.where(want > 3.4e38, torch.full_like(want, float("inf")), want)
        # bf16: 1 + 2^-8, of the fourth row's two values, is halfway between two numbers; fp32: values below
        # 2^-126 count as zero, so the sums lose 64 times 2^-128 of the other operand's
        off = 2.0 ** -8 * want.abs() if dt == torch.bfloat16 else torch.zeros_like(want)
        off[3] = torch.maximum(off[3], 64 * 2.0 ** -128 * b[:, 0].double())
        big = want.isinf()
        assert torch.equal(got[big], want[big])
        assert bool(((got - want).abs()[~big] <= off[~big] + 2.0 ** -126).all())


@pytest.mark.parametrize("out_dtype", DTYPES)
def test_empty_axes(out_dtype):
    a, b = mo.fp8_quantize(torch.zeros(5, 0, device="cuda")), mo.fp8_quantize(torch.zeros(7, 0, device="cuda"))
    out = torch.full((5, 9), 3.0, dtype=out_dtype, device="cuda")
    mo.fp8_matmul(a, b, out=out[:, 1:8])
    assert not out[:, 1:8].any() and bool((out[:, 0] == 3).all()) and bool((out[:, 8] == 3).all())
    out.fill_(3.0)
    mo.fp8_matmul(a, b, out=out[:, 1:8], accumulate=True)
    assert bool((out == 3).all())
    assert mo.fp8_matmul(mo.fp8_quantize(torch.zeros(0, 64, device="cuda")), mo.fp8_quantize(torch.ones(7, 64, device="cuda"))).shape == (0, 7)
    assert mo.fp8_dequantize(a).shape == (5, 0)


def test_product_of_many_rows():
    """More row tiles than a grid's second axis has places."""
    m = 64 * 65536 + 5
    a = torch.zeros(m, 2, device="cuda")
    a[:, 0] = torch.arange(m, device="cuda") % 7 - 3.0
    q = mo.fp8_quantize(a)
    got = mo.fp8_matmul(q, mo.fp8_quantize(torch.ones(1, 2, device="cuda")), out_dtype=torch.float32)
    assert torch.equal(got[:, 0], a[:, 0])


# --------------------------------------------------------------------- linear
@pytest.mark.parametrize("t,n,k", [(0, 40, 64), (1, 64, 96), (5, 33, 70), (130, 96, 257), (2, 300, 4100)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_and_backward(t, n, k, dtype):
    x, w = _rand((t, k), 1, dtype), _rand((n, k), 2, torch.float32, 0.05)
    dy = _rand((t, n), 3, dtype, 0.01)
    wq, wq_t = mo.fp8_quantize(w.cuda(), images="both", square=True)
    y, x_t = mo.fp8_linear(x.cuda(), wq, out_dtype=torch.float32, save=True)
    _check_product(y, of.rounded(_np(x)), of.rounded(_np(w), True), k)
    assert torch.equal(y, mo.fp8_linear(x.cuda(), wq, out_dtype=torch.float32))
    dx, dw = mo.fp8_linear_backward(dy.cuda(), x_t, wq_t, dx_dtype=torch.float32)
    _check_product(dx, of.rounded(_np(dy)), of.rounded(_np(w).T.copy(), True), n)
    _check_product(dw, of.rounded(_np(dy).T.copy()), of.rounded(_np(x).T.copy()), t)
    # two micro-batches into one gradient
    both = dw.clone()
    mo.fp8_linear_backward(dy.cuda(), x_t, wq_t, dw=both, accumulate=True)
    _check_product(both, of.rounded(_np(dy).T.copy()), of.rounded(_np(x).T.copy()), t, add=_np(dw))


def test_linear_keeps_leading_axes_and_empty_batches():
    w = mo.fp8_quantize(_rand((40, 64), 1, torch.float32).cuda())
    x = _rand((6, 64), 2, torch.bfloat16).cuda()
    y = mo.fp8_linear(x, w)
    assert torch.equal(mo.fp8_linear(x.view(2, 3, 64), w), y.view(2, 3, 40))
    assert mo.fp8_linear(x[:0], w).shape == (0, 40)
    assert mo.fp8_linear(x.view(2, 3, 64)[:0], w).shape == (0, 3, 40)


def test_refusals_leave_outputs_alone():
    x = _rand((40, 64), 1, torch.float32).cuda()
    q = mo.fp8_quantize(x)
    with pytest.raises(ValueError, match="expected an image"):
        mo.fp8_quantize(x, out=mo.Fp8Matrix.empty(40, 65, "cuda"))
    out = torch.full((40, 39), 2.0, device="cuda")
    with pytest.raises(ValueError, match="out must be"):
        mo.fp8_matmul(q, q, out=out)
    # an image whose codes lie inside the output
    big = torch.zeros(40 * 128 * 2, dtype=torch.uint8, device="cuda")
    inside = mo.Fp8Matrix(big[:q.codes.numel()].view(q.codes.shape), q.scales, 64)
    with pytest.raises(mo.MuonError, match="overlaps"):
        mo.fp8_matmul(inside, q, out=big[:3200].view(torch.bfloat16).view(40, 40))
    assert not bool(big.any())
    assert bool((out == 2.0).all())
    with pytest.raises(mo.MuonError, match="columns"):
        mo.fp8_matmul(q, mo.fp8_quantize(_rand((3, 65), 1, torch.float32).cuda()))


def test_optimizer_keeps_images():
    """Images of the matrices as they are behind each step, in place, with square scales."""
    ws = [_rand(s, i, torch.float32, 0.05).cuda() for i, s in enumerate([(130, 260), (64, 64)])]
    opt = mo.MuonAdamW(ws, lr=0.05, fp8="both", mx4="rows")
    first = opt.refresh_fp8()
    assert opt.refresh_fp8()[0][0] is first[0][0]
    for step in range(2):
        for i, w in enumerate(ws):
            w.grad = _rand(tuple(w.shape), 10 + i + step, torch.float32).cuda()
        opt.step()
        for w, (q, qt) in zip(ws, opt.fp8):
            _same_image(q, _np(w), True)
            _same_image(qt, _np(w).T.copy(), True)
    assert opt.fp8[0][0] is first[0][0] and len(opt.mx4) == 2
