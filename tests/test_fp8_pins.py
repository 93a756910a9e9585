"""The fp64 oracles of the 8-bit images, the cross entropy and the balance
loss against hand values, torch's e4m3 type and finite differences (CPU)."""

from __future__ import annotations

import numpy as np
import torch

from oracle import fp8 as of, linear_ce as oc


def test_table_is_e4m3():
    c = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(c, of.TABLE)


def test_scales_by_hand():
    # (largest magnitude, e)
    for a, e in [(448.0, 0), (np.nextafter(448.0, 500), 1), (1.0, -8), (1.75, -8), (np.nextafter(1.75, 2), -7), (0.0, -127),
                 (2.0 ** -149, -127), (448 * 2.0 ** -127, -127), (float(np.finfo(np.float32).max), 120), (np.inf, 128), (np.nan, 128)]:
        codes, scales = of.image(np.array([[a, 0.5 * a if np.isfinite(a) else 1.0]]))
        assert scales[0, 0] == e + 127, (a, e, scales[0, 0])
        assert codes.shape == (1, 128) and scales.shape == (1, 16) and not scales[0, 1:].any()
    # next to 2^128 a value stays below it
    assert of.rounded(np.array([[float(np.finfo(np.float32).max)]]))[0, 0] == 240 * 2.0 ** 120


def test_rounding_is_torchs():
    """Every bf16 value under a block's scale, against torch's conversion (which rounds to nearest even)."""
    g = np.random.default_rng(1)
    x = g.standard_normal((40, 256)) * np.exp2(g.integers(-12, 4, (40, 256)))
    codes, scales = of.image(x)
    t = x / np.exp2(np.repeat(scales[:, :2].astype(float), 128, axis=1) - 127)
    want = torch.from_numpy(t.astype(np.float32)).to(torch.float8_e4m3fn)
    assert np.array_equal(codes & 127, want.view(torch.uint8).numpy() & 127)
    assert np.max(np.abs(of.rounded(x) - x) / np.maximum(np.abs(x), 2.0 ** -6 * np.exp2(np.repeat(scales[:, :2].astype(float), 128, axis=1) - 127))) <= 2.0 ** -4


def test_square_images_transpose():
    # over many binades, so that some elements are subnormal under one scale and not under another
    g = np.random.default_rng(2)
    x = g.standard_normal((200, 300)) * np.exp2(g.integers(-20, 1, (200, 1))) * np.exp2(g.integers(-20, 1, (1, 300)))
    assert np.array_equal(of.rounded(x, True).T, of.rounded(x.T.copy(), True))
    assert not np.array_equal(of.rounded(x).T, of.rounded(x.T.copy()))


def test_cross_entropy_gradients_against_differences():
    gen = torch.Generator().manual_seed(3)
    x, w = (torch.randn(5, 7, generator=gen) * 2).bfloat16(), torch.randn(11, 7, generator=gen).bfloat16()
    t, g = torch.tensor([3, -1, 0, 10, 3]), torch.tensor([0.5, 2.0, 1.0, -0.25, 0.0])
    o = oc.cross_entropy(x, w, t, g)
    assert float(o.loss[1]) == 0 and not o.dx[1].any() and not o.dx[4].any()

    def total(xd, wd):
        z = xd @ wd.t()
        logp = torch.log_softmax(z, 1)
        return sum(float(g[i]) * -logp[i, t[i]] for i in range(5) if t[i] >= 0)

    xd, wd, h = x.double(), w.double(), 1e-6
    for m, d in ((xd, o.dx), (wd, o.dw)):
        for i in range(m.shape[0]):
            for j in range(m.shape[1]):
                keep = float(m[i, j])
                m[i, j] = keep + h
                up = total(xd, wd)
                m[i, j] = keep - h
                down = total(xd, wd)
                m[i, j] = keep
                # third derivatives of order 100, cancellation of values below 100 at 2^-52
                assert abs(float(up - down) / (2 * h) - float(d[i, j])) < 1e-7


def test_balance_gradient_against_differences():
    gen = torch.Generator().manual_seed(4)
    z = torch.randn(6, 5, generator=gen).double()
    idx = torch.tensor([[0, 1], [0, 0], [-1, -1], [4, -1], [2, 0], [0, 3]])
    loss, counts, grad = oc.balance(z, idx, 0.3, 2.0)
    assert counts.tolist() == [5, 1, 1, 1, 1] and not grad[2].any()
    h = 1e-6
    for i in range(6):
        for j in range(5):
            d = torch.zeros_like(z)
            d[i, j] = h
            diff = (oc.balance(z + d, idx, 0.3)[0] - oc.balance(z - d, idx, 0.3)[0]) / (2 * h)
            assert abs(2.0 * float(diff) - float(grad[i, j])) < 1e-8
    # perfect balance has the value of the weight
    even = torch.zeros(4, 2, dtype=torch.float64)
    assert abs(float(oc.balance(even, torch.tensor([[0], [1], [0], [1]]), 0.7)[0]) - 0.7) < 1e-15
