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


@pytest.mark.parametrize("k", [2049, 2176, 2200, 2432, 6273, 6528])
@pytest.mark.parametrize("tile", TILES)
def test_scales_that_end_inside_a_request(tile, k):
    """One to three stages into an odd group of sixteen, whole and partial:
    the place after the last scale dword is then the end of the kernel's
    shared memory, which nothing may read."""
    if tile == "256" and k > 2432:
        pytest.skip("the same place as the shorter ones, and a long oracle")
    m, n = TILES[tile]
    a, b, av, bv = _images(m, n, k)
    for dt in DTYPES:
        _check_product(mo.mx4_matmul(a, b, out_dtype=dt), av, bv, k)
