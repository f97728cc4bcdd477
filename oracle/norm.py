"""Residual addition with the root-mean-square norm, and its gradients, in fp64.

TEST INFRASTRUCTURE ONLY: see ``oracle/__init__.py`` for who may import this.

    h = RN16(RN32(x + res)),  rstd = (mean(h^2) + eps)^-1/2,  y = h rstd w
    L's gradients from dy = dL/dy and dres = dL/dh past the norm:
    dx = rstd (g - hn mean(g hn)) + dres,  g = dy w,  hn = h rstd;   dw = sum_m dy hn

The stream h is rounded before it is normalised (the backward reads it again);
everything after it is exact here. The error bounds count the roundings of an
fp32 evaluation: ``depth`` additions in a chain for a sum over a row or over
the rows, one unit (2^-24) for every other operation.
"""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def rms_fwd(h, w, eps: float):
    """(y, rstd) of the stream h [M, k] and the gain w [k]."""
    h, w = np.asarray(h, dtype=np.float64), np.asarray(w, dtype=np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * w, rstd


def rms_bwd(dy, h, rstd, w, dres=None):
    """(dx, dw) with rstd as it was saved."""
    dy, h, rstd, w = (np.asarray(a, dtype=np.float64) for a in (dy, h, rstd, w))
    hn = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - hn * (g * hn).mean(axis=1, keepdims=True))
    return dx if dres is None else dx + np.asarray(dres, dtype=np.float64), (dy * hn).sum(axis=0)


def rstd_bound(k: int) -> float:
    """Relative error of rstd: the chain of a row's sum (squares of 16-bit values are exact in fp32: three additions
    of eight, a thread's eights, 4 + 2 across the wave; the waves' sums, the mean and eps are fp64), halved by the
    square root, eps as fp32 (half a step of at most the whole) and one rounding."""
    return ((3 + max(4, -(-k // 8192)) + 6 + 1) / 2 + 1.01) * U


def row_depth(k: int) -> int:
    """Additions in a chain of a row's sum: at most 32 values of a thread (more where 1024 threads hold less than the
    row), 4 + 2 across the wave, 16 waves."""
    return 8 * max(4, -(-k // 8192)) + 22


def y_bound(y, k: int, u16: float, tiny: float):
    """Error of y: rstd's and two products, then half a step of 16 bits (tiny: half the type's smallest step)."""
    e = np.abs(y) * (rstd_bound(k) + 2 * U)
    return e + u16 * (np.abs(y) + e) + tiny


def dx_bound(dy, h, rstd, w, dres, dx, u16: float, tiny: float):
    """Error of dx: every term of its sum with the roundings before it, then half a step of 16 bits."""
    dy, h, rstd, w = (np.asarray(a, dtype=np.float64) for a in (dy, h, rstd, w))
    hn, g = h * rstd[:, None], dy * w
    s = np.abs(rstd)[:, None] * (np.abs(g) + np.abs(hn) * np.abs(g * hn).mean(axis=1, keepdims=True))
    if dres is not None:
        s = s + np.abs(np.asarray(dres, dtype=np.float64))
    e = (row_depth(h.shape[1]) + 10) * U * s
    return e + u16 * (np.abs(dx) + e) + tiny


def dw_bound(dy, h, rstd):
    """Error of dw: its chain is a thread's rows (at most ceil(M / 64), at least 64 workgroups walk over them), up to
    64 rows of a workgroup, and 16 + 16 partial sums."""
    dy, h, rstd = (np.asarray(a, dtype=np.float64) for a in (dy, h, rstd))
    depth = -(-h.shape[0] // 64) + 64 + 32
    return (depth + 3) * U * np.abs(dy * h * rstd[:, None]).sum(axis=0)
