"""Products of MX4 images by the kernel that computes them: lengths at which
the scale bytes end inside a request of the tile kernel, in tiles of every
size.  Oracle and tolerances are those of test_mx4_gpu.
"""

from __future__ import annotations

import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from test_mx4_gpu import DTYPES, _check_product, _np, _rand

pytestmark = pytest.mark.gpu

# rows of a and b that take each tile size
TILES = {"64": (70, 100), "128": (1500, 1700), "256": (3900, 3301)}


def _images(m, n, k):
    a, b = mo.mx4_quantize(_rand((m, k), m + k, torch.float32).cuda()), mo.mx4_quantize(_rand((n, k), n + k, torch.bfloat16).cuda())
    return a, b, _np(mo.mx4_dequantize(a, dtype=torch.float32)), _np(mo.mx4_dequantize(b, dtype=torch.float32))


# (the longer ones reach the same place as the shorter, at a long oracle's cost in the largest tile)
@pytest.mark.parametrize("tile,k", [(t, k) for t in TILES for k in (2049, 2176, 2200, 2432, 6273, 6528)
                                    if t != "256" or k <= 2432])
def test_scales_that_end_inside_a_request(tile, k):
    """One to three stages into an odd group of sixteen, whole and partial:
    the place after the last scale dword is then the end of the kernel's
    shared memory, which nothing may read."""
    m, n = TILES[tile]
    a, b, av, bv = _images(m, n, k)
    for dt in DTYPES:
        _check_product(mo.mx4_matmul(a, b, out_dtype=dt), av, bv, k)


# rows of a and b and a contraction that take each kernel
KERNELS = {"skinny": (5, 170, 700), "direct": (200, 300, 200), "64": (130, 257, 700), "128": (1500, 1700, 520),
           "256": (3900, 3301, 520)}


@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("kernel", KERNELS)
def test_accumulates_into_strided_rows(kernel, out_dtype):
    """Adds to rows that start anywhere; the columns between them stay."""
    m, n, k = KERNELS[kernel]
    a, b, av, bv = _images(m, n, k)
    for pad, off in ((0, 0), (2, 1)):
        buf = _rand((m, n + pad + off), 3, out_dtype, 50.0).cuda()
        keep = buf.clone()
        out = buf[:, off:off + n]
        add = _np(out)
        assert mo.mx4_matmul(a, b, out=out, accumulate=True) is out
        _check_product(out, av, bv, k, add)
        keep[:, off:off + n] = out
        assert torch.equal(buf, keep)


@pytest.mark.parametrize("kernel", KERNELS)
def test_nan_blocks_and_wide_scales(kernel):
    """Blocks of NaN or infinities, the last and the first one among them, make
    their rows or columns NaN and nothing else; scales from 2^-60 to 2^60."""
    m, n, k = KERNELS[kernel]
    g = torch.Generator().manual_seed(5)
    a = torch.randn(m, k, generator=g) * torch.exp2(torch.linspace(-60, 60, k))
    b = torch.randn(n, k, generator=g) * torch.exp2(torch.linspace(50, -70, k))
    a[3, k - 1], a[m - 1, 40], b[n - 2, 0], b[2, k // 2] = float("nan"), float("inf"), -float("inf"), float("nan")
    qa, qb = mo.mx4_quantize(a.cuda()), mo.mx4_quantize(b.cuda())
    av, bv = _np(mo.mx4_dequantize(qa, dtype=torch.float32)), _np(mo.mx4_dequantize(qb, dtype=torch.float32))
    got = mo.mx4_matmul(qa, qb, out_dtype=torch.float32)
    nan = torch.zeros(m, n, dtype=torch.bool)
    nan[[3, m - 1]] = True
    nan[:, [n - 2, 2]] = True
    assert torch.equal(torch.isnan(got).cpu(), nan)
    _check_product(got, av, bv, k)
