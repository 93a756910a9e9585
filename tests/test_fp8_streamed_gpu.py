"""Products of 8-bit images whose outputs go past the caches: more than 32 MiB
in whole lines, written and added to, beside ones of the same size that do not."""

from __future__ import annotations

import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from test_fp8_gpu import DTYPES, _check_product, _np, _rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(4100, 4160, 200), (1030, 16448, 130), (70, 262144, 128)])
def test_outputs_past_the_caches(m, n, k, out_dtype):
    a, b = mo.fp8_quantize(_rand((m, k), 1, torch.float32).cuda()), mo.fp8_quantize(_rand((n, k), 2, torch.float32).cuda())
    av, bv = _np(mo.fp8_dequantize(a, dtype=torch.float32)), _np(mo.fp8_dequantize(b, dtype=torch.float32))
    got = mo.fp8_matmul(a, b, out_dtype=out_dtype)
    assert got.numel() * got.element_size() > 32 << 20 and got.data_ptr() % 128 == 0 and n * got.element_size() % 128 == 0
    _check_product(got, av, bv, k)
    out = _rand((m, n), 3, out_dtype, 50.0).cuda()
    add = _np(out)
    assert mo.fp8_matmul(a, b, out=out, accumulate=True) is out
    _check_product(out, av, bv, k, add)
    # rows a line apart: the same lines, and what lies between stays as it was
    buf = torch.full((m, n + 256 // got.element_size()), 7.0, dtype=out_dtype, device="cuda")
    mo.fp8_matmul(a, b, out=buf[:, :n])
    assert torch.equal(buf[:, :n], got) and bool((buf[:, n:] == 7).all())
    # rows that share lines: through the caches, the same bits
    buf = torch.full((m, n + 3), 7.0, dtype=out_dtype, device="cuda")
    mo.fp8_matmul(a, b, out=buf[:, :n])
    assert torch.equal(buf[:, :n], got) and bool((buf[:, n:] == 7).all())
