"""fp64 oracle of the 8-bit (e4m3, a power of two per block of 128) images.

Definitions of ``include/muon.h`` in numpy fp64: every value of an image is
exact there.
"""

from __future__ import annotations

import numpy as np

BLOCK = 128
#: the 127 magnitudes, by code
TABLE = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])


def _blocks(x: np.ndarray, square: bool) -> np.ndarray:
    """[row blocks, rows of one, column blocks, 128], padded with zeros."""
    r, c = x.shape
    k = BLOCK if square else 1
    p = np.zeros((-(-r // k) * k, -(-c // BLOCK) * BLOCK))
    p[:r, :c] = x
    return p.reshape(p.shape[0] // k, k, -1, BLOCK)


def _scale(a: np.ndarray) -> np.ndarray:
    """The smallest e with a <= 448 2^e, at least -127; 128 for NaN and infinity."""
    out = np.full(a.shape, -127)
    for i, v in np.ndenumerate(a):
        if not np.isfinite(v):
            out[i] = 128
        elif v > 0:
            m, e = np.frexp(v)                       # 448 = 0.875 2^9
            out[i] = max(-127, int(e) - 9 + (m > 0.875))
    return out


def _codes(t: np.ndarray, e: np.ndarray) -> np.ndarray:
    """Codes of scaled elements: the nearer of two neighbours, halves to the even code."""
    m = np.abs(t)
    hi = np.clip(np.searchsorted(TABLE, m), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, up = m - TABLE[lo], TABLE[hi] - m
    c = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    c = np.where((e == 120) & (TABLE[c] > 240), np.searchsorted(TABLE, 240.0), c)     # 2^128 is past fp32
    return (c | (np.signbit(t) * 128)).astype(np.uint8)


def image(x: np.ndarray, square: bool = False):
    """(codes uint8 [r, 128 nb], scales uint8 [r, 16 ceil(nb / 16)]) of fp64 [r, c]."""
    r = x.shape[0]
    if x.size == 0:
        nb = -(-x.shape[1] // BLOCK)
        return np.zeros((r, nb * BLOCK), np.uint8), np.zeros((r, -(-nb // 16) * 16), np.uint8)
    b = _blocks(np.asarray(x, np.float64), square)
    with np.errstate(invalid="ignore"):
        a = np.max(np.abs(b), axis=(1, 3), keepdims=True)
    e = _scale(a)
    with np.errstate(invalid="ignore", over="ignore"):
        codes = np.where(e == 128, 0, _codes(np.where(e == 128, 0.0, b) * np.exp2(-e.astype(float)), e)).astype(np.uint8)
    nb = b.shape[2]
    scales = np.zeros((b.shape[0] * b.shape[1], -(-nb // 16) * 16), np.uint8)
    scales[:, :nb] = np.broadcast_to(e, b.shape)[:, :, :, 0].reshape(-1, nb) + 127
    return codes.reshape(-1, nb * BLOCK)[:r], scales[:r]


def values(codes: np.ndarray, scales: np.ndarray, cols: int) -> np.ndarray:
    """What an image stands for."""
    v = np.append(TABLE, np.nan)[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(float) - 127.0))
    return (v * np.repeat(s, BLOCK, axis=1)[:, :v.shape[1]])[:, :cols]


def rounded(x: np.ndarray, square: bool = False) -> np.ndarray:
    return values(*image(x, square), x.shape[1])
