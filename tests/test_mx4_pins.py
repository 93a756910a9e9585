"""Pins of the MX4 and distillation oracles on the CPU: the rounding against
the full list of halfway cases, blocks whose images are known by hand, and
the distillation gradient against central differences of its loss."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import distill as od, mx4 as om

HALFWAY = {0.25: 0.0, 0.75: 1.0, 1.25: 1.0, 1.75: 2.0, 2.5: 2.0, 3.5: 4.0, 5.0: 4.0}


def test_rounding_of_every_halfway_case():
    for x, want in HALFWAY.items():
        for eps, w in ((0.0, want),
                       (-1e-9, max(v for v in om.GRID if v <= x)),
                       (1e-9, min(v for v in om.GRID if v >= x))):
            assert om.GRID[om.nearest_code(np.array([x + eps]))[0]] == w, (x, eps)
    assert om.GRID[om.nearest_code(np.array([7.99]))[0]] == 6.0


def test_known_blocks():
    x = np.zeros((1, 40))
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 4.0, -1.0, 0.25, 6.5
    x[0, 32] = 2.0 ** -10
    codes, scales = om.image(x)
    assert scales.tolist() == [[127, 127 - 12, 0, 0]]
    assert codes[0, 0] == 6 | (2 | 8) << 4 and codes[0, 1] == 0 | 7 << 4
    assert codes[0, 16] == 6
    assert om.values((codes, scales), 40)[0, :4].tolist() == [4.0, -1.0, 0.0, 6.0]


def test_zero_nan_and_tiny_blocks():
    x = np.zeros((3, 32))
    x[1, 5] = np.inf
    x[2, 0], x[2, 1] = 2.0 ** -140, -(2.0 ** -128)
    codes, scales = om.image(x)
    assert scales[:, 0].tolist() == [0, 255, 0]
    assert not codes[:2].any()
    v = om.values((codes, scales), 32)
    assert np.isnan(v[1]).all() and v[2, 0] == 0.0 and v[2, 1] == -(2.0 ** -128)


def test_values_round_to_themselves():
    rng = np.random.default_rng(0)
    v = om.rounded(rng.standard_normal((5, 70)))
    # a block whose largest value rounds to 4 or 6 keeps its scale
    assert np.array_equal(om.rounded(v), v)


@pytest.mark.parametrize("tau", [1.0, 0.5, 3.0])
def test_distill_gradient_against_differences(tau):
    rng = np.random.default_rng(1)
    z = rng.standard_normal((4, 23))
    idx = np.array([[1, 5, 7], [2, 2, 9], [22, -1, 0], [-1, -1, -1]])
    t = rng.standard_normal((4, 3)).astype(np.float32)
    g = np.array([1.0, -0.5, 2.0, 1.0])
    _, grad = od.distill(z, idx, t, tau, g)
    h = 1e-4
    for j in range(z.shape[1]):
        up, dn = z.copy(), z.copy()
        up[:, j] += h
        dn[:, j] -= h
        num = g * (od.distill(up, idx, t, tau)[0] - od.distill(dn, idx, t, tau)[0]) / (2 * h)
        # central differences: h^2 / 6 of a third derivative below 2 / tau,
        # and rounding of the losses over h
        assert np.all(np.abs(num - grad[:, j]) <= 1e-8 / tau + 1e-9)
    assert not grad[3].any()


def test_distill_of_one_slot_is_cross_entropy():
    rng = np.random.default_rng(2)
    z = rng.standard_normal((6, 31))
    lab = rng.integers(0, 31, (6, 1))
    loss, _ = od.distill(z, lab, np.zeros((6, 1), np.float32))
    lse = np.log(np.exp(z).sum(1))
    assert np.allclose(loss, lse - z[np.arange(6), lab[:, 0]], rtol=1e-13)


def test_logprobs_order_and_entropy():
    z = np.array([[1.0, 3.0, 3.0, -np.inf, 0.0], [np.nan, 1.0, np.inf, 2.0, -0.0]])
    lp, ent, tlp, tix = od.token_logprobs(z, np.array([0, 1]), 5)
    assert tix.tolist() == [[1, 2, 0, 4, 3], [0, 2, 3, 1, 4]]
    p = np.exp([1.0, 3.0, 3.0, 0.0])
    p /= p.sum()
    assert abs(ent[0] + (p * np.log(p)).sum()) < 1e-14 and np.isnan(ent[1]) and np.isnan(lp[1])
    assert tlp[0, 4] == -np.inf
