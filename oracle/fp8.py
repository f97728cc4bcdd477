"""The 8-bit layer in fp64: block scales, E4M3 rounding, and the layer over
the encoded values.

TEST INFRASTRUCTURE ONLY: see ``oracle/__init__.py`` for who may import this.

An E4M3 value has 4 exponent bits of bias 7 and 3 mantissa bits, subnormals in
steps of 2^-9, largest finite 448, one NaN pattern per sign and no infinity. A
block of 128 (of one row for activations, a 128 x 128 tile for weights) shares
a scale 2^(b - 127): the smallest whole b >= 0 with max |x| <= 448 2^(b - 127),
127 for a block without nonzero finite values. An element is stored as the
E4M3 value nearest x / scale, ties to the even code, NaN where x is not finite.

    Y  = X8 W8^T + s (X A^T) B^T
    dX = dY8 W8 + s U A,  dA = s U^T X,  dB = s dY^T (X A^T),  U = dY B
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

BLOCK = 128


def table() -> np.ndarray:
    """The 256 values by code, NaN at 0x7F and 0xFF."""
    t = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if b & 0x7F == 0x7F:
            v = np.nan
        t[b] = -v if b & 0x80 else v
    return t


def scale_byte(amax: float) -> int:
    """Exponent byte of a block whose largest finite magnitude is amax."""
    if amax == 0:
        return 127
    b = 0
    while Fraction(float(amax)) > 448 * Fraction(2) ** (b - 127):
        b += 1
    return b


def _bytes_of(amax: np.ndarray) -> np.ndarray:
    u, inv = np.unique(amax, return_inverse=True)
    return np.array([scale_byte(a) for a in u], dtype=np.uint8)[inv].reshape(amax.shape)


def encode_values(v) -> np.ndarray:
    """Codes of v (already divided by its scale, |v| <= 448 or not finite)."""
    v = np.asarray(v, dtype=np.float64)
    pos = table()[:127]
    a = np.where(np.isfinite(v), np.abs(v), 0.0)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)          # first value >= a
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - pos[lo], pos[hi] - a
    c = np.where((dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0)), hi, lo)
    c = np.where(np.isfinite(v), c, 0x7F)
    return (c | (np.signbit(v) << 7)).astype(np.uint8)


def _finite_max(x, axis):
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    return a.max(axis=axis, keepdims=True)


def encode_rows(X):
    """(codes [M, Cp], bytes [M, Cp / 128]) of activations."""
    X = np.asarray(X, dtype=np.float64)
    M, C = X.shape
    p = np.zeros((M, -(-C // BLOCK) * BLOCK))
    p[:, :C] = X
    p = p.reshape(M, -1, BLOCK)
    b = _bytes_of(_finite_max(p, 2))
    with np.errstate(invalid="ignore"):
        codes = encode_values(p / np.ldexp(1.0, b.astype(int) - 127))
    return codes.reshape(M, -1), b[:, :, 0]


def encode_weight(W):
    """(codes [n, kp], bytes [ceil(n / 128), kp / 128]) of a weight."""
    W = np.asarray(W, dtype=np.float64)
    n, k = W.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    p = np.zeros((nb * BLOCK, kb * BLOCK))
    p[:n, :k] = W
    p = p.reshape(nb, BLOCK, kb, BLOCK)
    b = _bytes_of(_finite_max(p, (1, 3)))
    with np.errstate(invalid="ignore"):
        codes = encode_values(p / np.ldexp(1.0, b.astype(int) - 127))
    return codes.reshape(nb * BLOCK, kb * BLOCK)[:n], b[:, 0, :, 0]


def rows_values(codes, b, C) -> np.ndarray:
    v = table()[codes] * np.repeat(np.ldexp(1.0, b.astype(int) - 127), BLOCK, axis=1)
    return v[:, :C]


def weight_values(codes, b, n, k) -> np.ndarray:
    s = np.ldexp(1.0, b.astype(int) - 127)
    return (table()[codes] * np.repeat(np.repeat(s, BLOCK, 0)[:n], BLOCK, 1))[:, :k]


def linear_fwd(X, W8, A, B, s):
    """(Y, T) over the weight values W8, X encoded by row blocks."""
    X = np.asarray(X, dtype=np.float64)
    Y = rows_values(*encode_rows(X), X.shape[1]) @ W8.T
    if A is None:
        return Y, None
    T = X @ np.asarray(A, dtype=np.float64).T
    return Y + s * (T @ np.asarray(B, dtype=np.float64).T), T


def linear_bwd(X, W8, A, B, s, dY):
    """(dX, dA, dB) over the weight values W8, dY encoded by row blocks for dX."""
    X, dY = np.asarray(X, dtype=np.float64), np.asarray(dY, dtype=np.float64)
    dX = rows_values(*encode_rows(dY), dY.shape[1]) @ W8
    if A is None:
        return dX, None, None
    A, B = np.asarray(A, dtype=np.float64), np.asarray(B, dtype=np.float64)
    U = dY @ B
    return dX + s * (U @ A), s * (U.T @ X), s * (dY.T @ (X @ A.T))
