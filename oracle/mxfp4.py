"""MXFP4 in float64, from the format's definition.

TEST INFRASTRUCTURE ONLY (see the package docstring).

* Elements E2M1, two to a byte, element 2j of a row in the low nibble of byte j; one E8M0 scale byte s
  per 32 elements of a row: E2M1(code) * 2^(s - 127), NaN for s = 255.
* Nearest (OCP MX v1.0): X = clamp(floor(log2 amax) - 2, -127, 127), elements x / 2^X rounded half to
  even on the E2M1 grid, saturating at 6.  Stochastic: X = the least exponent >= -127 with
  amax <= 6 * 2^X, and |code| = step * floor((floor(v / step * 2^16) + r) / 2^16).
* A negative element that rounds to zero is -0; a block of zeros is scale 0 and codes 0; a block with an
  infinity or a NaN is scale 255 and codes 0.  Rows are padded with zeros to whole blocks.
* The draws are Philox4x32 (Salmon et al. 2011) with 7 rounds: element i of the row-major matrix takes
  half word i % 8 (low halves first) at counter i // 8.
"""
from __future__ import annotations

import numpy as np

from .numerics import E2M1_TABLE, e8m0_to_f64

BLOCK = 32


def philox4x32(counter, key, rounds):
    """Four words for each 64-bit counter (the upper two counter words are zero), uint64 [n, 4]."""
    low = np.uint64(0xFFFFFFFF)
    n = np.asarray(counter, dtype=np.uint64)
    c = [n & low, n >> np.uint64(32), np.zeros_like(n), np.zeros_like(n)]
    k0, k1 = int(key) & 0xFFFFFFFF, (int(key) >> 32) & 0xFFFFFFFF
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & low, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1)


def draws(rows, cols, key):
    """The 16-bit draws of a [rows, cols] matrix, int64."""
    n = rows * cols
    w = philox4x32(np.arange((n + 7) // 8), key, 7)
    half = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(-1)
    return half[:n].astype(np.int64).reshape(rows, cols)


def _padded(x):
    r, c = x.shape
    out = np.zeros((r, -(-c // BLOCK) * BLOCK), x.dtype)
    out[:, :c] = x
    return out


def quantize(x, r=None):
    """(packed codes [R, Cp/2], scales [R, Cp/32]) of real x [R, C]; r: draws [R, C], or None for nearest."""
    x = _padded(np.asarray(x, dtype=np.float64))
    rows, k = x.shape
    b = x.reshape(rows, k // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    zero = amax == 0
    m, e = np.frexp(np.where(zero, 1.0, amax))               # amax = m 2^e, m in [0.5, 1)
    X = e - 1 - 2 if r is None else e - 1 - 2 + (m > 0.75)
    X = np.clip(X, -127, 127)
    v = np.abs(b) / np.exp2(X)[..., None]
    step = np.where(v < 2, 0.5, np.where(v < 4, 1.0, 2.0))
    if r is None:
        mag = np.minimum(np.rint(v / step) * step, 6.0)
    else:
        d = _padded(np.asarray(r, dtype=np.int64)).reshape(b.shape)
        mag = np.floor((np.floor(v / step * 65536) + d) / 65536) * step
    codes = np.searchsorted(E2M1_TABLE[:8], mag)
    assert np.array_equal(E2M1_TABLE[codes], mag)
    codes = codes | np.where(np.signbit(b), 8, 0)
    codes = np.where((zero | bad)[..., None], 0, codes).reshape(rows, k).astype(np.uint8)
    scales = np.where(bad, 255, np.where(zero, 0, X + 127)).astype(np.uint8)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def dequantize(packed, scales):
    packed = np.asarray(packed, dtype=np.uint8)
    rows, half = packed.shape
    codes = np.empty((rows, 2 * half), np.uint8)
    codes[:, 0::2], codes[:, 1::2] = packed & 15, packed >> 4
    v = E2M1_TABLE[codes].reshape(rows, -1, BLOCK) * e8m0_to_f64(scales)[..., None]
    return v.reshape(rows, 2 * half)


def product(a, b):
    """deq(a) . deq(b)^T and sum |deq(a)| |deq(b)| of (codes, scales) pairs or real matrices."""
    a, b = (dequantize(*m) if isinstance(m, tuple) else np.asarray(m, dtype=np.float64) for m in (a, b))
    return a @ b.T, np.abs(a) @ np.abs(b).T
