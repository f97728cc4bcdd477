"""Pins of oracle/norm.py and of the clip factor: closed forms, fp64 autograd and central differences."""

import numpy as np
import pytest
import torch

from oracle import adamw as oadam
from oracle import norm as onorm


def _draw(M, k, seed=0):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((M, k)), rng.standard_normal(k), rng.standard_normal((M, k)), rng.standard_normal((M, k))


def test_closed_forms():
    y, rstd = onorm.rms_fwd([[3.0, -4.0]], [1.0, 2.0], 0.0)
    assert rstd[0] == pytest.approx(1 / np.sqrt(12.5), rel=1e-15)
    assert y[0] == pytest.approx([3 / np.sqrt(12.5), -8 / np.sqrt(12.5)], rel=1e-15)
    y, rstd = onorm.rms_fwd(np.zeros((2, 5)), np.ones(5), 1e-4)
    assert np.all(y == 0) and rstd == pytest.approx([100.0, 100.0])
    # one column, eps 0: y is the sign times the gain, and no gradient passes
    y, rstd = onorm.rms_fwd([[-7.0]], [3.0], 0.0)
    assert y[0, 0] == pytest.approx(-3.0)
    dx, dw = onorm.rms_bwd([[2.0]], [[-7.0]], rstd, [3.0])
    assert abs(dx[0, 0]) < 1e-15 and dw[0] == pytest.approx(-2.0)


@pytest.mark.parametrize("M,k", [(1, 1), (3, 7), (5, 64)])
def test_gradients_by_autograd_and_differences(M, k):
    h, w, dy, dres = _draw(M, k, k)
    _, rstd = onorm.rms_fwd(h, w, 1e-3)
    dx, dw = onorm.rms_bwd(dy, h, rstd, w, dres)
    ht, wt = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = ht * torch.rsqrt((ht * ht).mean(1, keepdim=True) + 1e-3) * wt
    ((y * torch.tensor(dy)).sum() + (ht * torch.tensor(dres)).sum()).backward()
    assert np.allclose(dx, ht.grad.numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(dw, wt.grad.numpy(), rtol=1e-12, atol=1e-13)
    L = lambda h, w: float((onorm.rms_fwd(h, w, 1e-3)[0] * dy).sum() + (h * dres).sum())  # noqa: E731
    rng = np.random.default_rng(5)
    vh, vw, e = rng.standard_normal((M, k)), rng.standard_normal(k), 1e-6
    num = (L(h + e * vh, w + e * vw) - L(h - e * vh, w - e * vw)) / (2 * e)
    assert num == pytest.approx(float((dx * vh).sum() + (dw * vw).sum()), rel=1e-6, abs=1e-7)


def test_bounds_hold_for_fp32_sums_and_catch_a_wrong_value():
    h, w, dy, dres = (a.astype(np.float32) for a in _draw(40, 300, 3))
    y, rstd = onorm.rms_fwd(h, w, 1e-5)
    r32 = (1 / np.sqrt((h * h).cumsum(axis=1, dtype=np.float32)[:, -1] / np.float32(300) + np.float32(1e-5))).astype(np.float32)
    # (a chain of 300 additions where the kernels have row_depth: its own depth instead)
    assert np.all(np.abs(r32 - rstd) <= rstd * (300 / 2 + 4) * onorm.U)
    t = torch.tensor(h * r32[:, None] * w).bfloat16().double().numpy()
    wide = np.abs(y) * 300 * onorm.U
    assert np.all(np.abs(t - y) <= onorm.y_bound(y, 300, 2.0 ** -8, 0) + wide)
    assert np.any(np.abs(t * (1 + 2.0 ** -7) - y) > onorm.y_bound(y, 300, 2.0 ** -8, 0) + wide)
    dx, dw = onorm.rms_bwd(dy, h, rstd, w, dres)
    b = onorm.dx_bound(dy, h, rstd, w, dres, dx, 2.0 ** -8, 0)
    assert np.all(np.abs(torch.tensor(dx).bfloat16().double().numpy() - dx) <= b)
    lost, _ = onorm.rms_bwd(dy, h, rstd, w, None)
    assert np.any(np.abs(lost - dx) > b)
    part, _ = onorm.rms_bwd(dy[:, :-1], h[:, :-1], rstd, w[:-1], dres[:, :-1])  # a mean over too few columns
    assert np.any(np.abs(part - dx[:, :-1]) > b[:, :-1])
    _, less = onorm.rms_bwd(dy[:-1], h[:-1], rstd[:-1], w)
    assert np.any(np.abs(less - dw) > onorm.dw_bound(dy, h, rstd))


def test_clip_factor():
    a, b = np.array([3.0, 0.0]), np.array([[4.0]])
    assert oadam.clip_factor([a, b], 10.0) == (5.0, 1.0)
    assert oadam.clip_factor([a, b], 2.5) == (5.0, 0.5)
    assert oadam.clip_factor([a, b], 1.0, 0.5) == (2.5, 0.4)
    assert oadam.clip_factor([], 1.0) == (0.0, 1.0)
    g = torch.nn.Parameter(torch.zeros(3))
    g.grad = torch.tensor([3.0, 0.0, 4.0])
    assert float(torch.nn.utils.clip_grad_norm_([g], 2.5)) == 5.0
    assert g.grad.numpy() == pytest.approx(np.array([3.0, 0.0, 4.0]) * oadam.clip_factor([a, b], 2.5)[1], rel=1e-6)
    for bad in (np.inf, -np.inf, np.nan):
        norm, f = oadam.clip_factor([a, np.array([bad])], 1.0)
        assert not np.isfinite(norm) and np.isnan(f)
