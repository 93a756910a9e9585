"""fp64 oracle of the MX4 format: quantisation, images, values, products.

Written from the format's definition: 32 consecutive elements of a row share
a power of two, an element is a sign and one of eight magnitudes.  The
rounding searches the list of magnitudes; nothing is shared with the kernels.
"""

from __future__ import annotations

import math

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks(cols: int) -> int:
    return -(-cols // 32)


def nearest_code(t: np.ndarray) -> np.ndarray:
    """Index of the nearest magnitude of |t|, the even one of two equally
    near, the last one above the list."""
    m = np.abs(t)
    dist = np.abs(m[..., None] - GRID)
    best = dist.min(-1, keepdims=True)
    near = dist == best                       # at most two neighbours
    first = near.argmax(-1)
    second = 7 - near[..., ::-1].argmax(-1)
    return np.where(first % 2 == 0, first, second).astype(np.uint8)


def quantize(x: np.ndarray):
    """(codes [rows, 32 nb], scale bytes [rows, nb]) of an exact fp64 array."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = blocks(cols)
    p = np.zeros((rows, nb * 32))
    p[:, :cols] = x
    codes = np.zeros((rows, nb * 32), np.uint8)
    scales = np.zeros((rows, nb), np.uint8)
    for r in range(rows):
        for b in range(nb):
            v = p[r, 32 * b:32 * b + 32]
            if not np.all(np.isfinite(v)):
                scales[r, b] = 255
                continue
            a = float(np.max(np.abs(v)))
            e = -127 if a == 0.0 else max(math.frexp(a)[1] - 3, -127)   # floor(log2 a) - 2
            scales[r, b] = e + 127
            c = nearest_code(v * 2.0 ** -e)
            n = min(32, cols - 32 * b)
            c[:n] |= np.where(np.signbit(v[:n]), 8, 0).astype(np.uint8)
            codes[r, 32 * b:32 * b + 32] = c
    return codes, scales


def image(x: np.ndarray):
    """The stored arrays (codes [rows, 16 nb], scales [rows, 4 ceil(nb / 4)])."""
    codes, s = quantize(x)
    rows, nb = s.shape
    scales = np.zeros((rows, -(-nb // 4) * 4), np.uint8)
    scales[:, :nb] = s
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def values(stored, cols: int) -> np.ndarray:
    """What stored arrays stand for, fp64 [rows, cols]."""
    packed, scales = stored
    rows = packed.shape[0]
    codes = np.zeros((rows, packed.shape[1] * 2), np.uint8)
    codes[:, 0::2] = packed & 15
    codes[:, 1::2] = packed >> 4
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.ldexp(1.0, scales.astype(np.int64) - 127)
    s = np.where(scales == 255, np.nan, s)
    return (v * np.repeat(s, 32, axis=1)[:, :v.shape[1]])[:, :cols]


def rounded(x: np.ndarray) -> np.ndarray:
    """The values of x's image."""
    return values(image(x), x.shape[1])
