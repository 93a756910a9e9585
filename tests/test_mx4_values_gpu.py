"""The 4-bit rounding of every bf16 value, at every distance from its block's
largest one that tells it from zero, against the oracle's search."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from oracle import mx4 as om

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("above", [None, 0, 1, 2, 3, 4])
def test_every_bf16_value(above, dtype):
    """Row r of [65536, 2] holds the value with bit pattern r, alone or beside
    a power of two `above` binades over it."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v64 = v.double().numpy()
    finite = np.isfinite(v64)
    mag = np.where(finite, np.abs(v64), 1.0)
    top = np.zeros(65536)
    if above is not None:
        lead = np.where(mag > 0, np.frexp(mag)[1] - 1, 0)
        top = np.ldexp(1.0, np.clip(lead + above, -133, 127))
    x = torch.stack([v, torch.from_numpy(top).to(torch.bfloat16)], 1)
    assert np.array_equal(x[:, 1].double().numpy(), top)
    q = mo.mx4_quantize(x.to(dtype).cuda())
    a = np.maximum(mag, top)
    e = np.where(a > 0, np.maximum(np.frexp(a)[1] - 3, -127), -127)      # floor(log2 a) - 2
    scales = np.where(finite, e + 127, 255).astype(np.uint8)
    code = [om.nearest_code(np.ldexp(np.where(finite, t, 0.0), -e)) for t in (v64, top)]
    code[0] |= np.where(finite & np.signbit(v64), 8, 0).astype(np.uint8)
    code[1] = np.where(finite, code[1], 0).astype(np.uint8)
    assert np.array_equal(q.scales[:, 0].cpu().numpy(), scales)
    assert np.array_equal(q.codes[:, 0].cpu().numpy(), code[0] | code[1] << 4)
    assert not bool(q.codes[:, 1:].any()) and not bool(q.scales[:, 1:].any())
    # the same values down a column
    t = mo.mx4_quantize(x.to(dtype).t().contiguous().cuda(), images="cols")
    assert torch.equal(t.codes, q.codes) and torch.equal(t.scales, q.scales)
