"""The norm at the ends of fp32's range (qlora_rms_norm_fwd, qlora_rms_norm_bwd): rows whose squares overflow or vanish, gains far from one.

y is RN16 of two fp32 products of h, rstd and w. Each rounds by 2^-24 of its value or, among the smallest numbers, by
2^-150; a factor that is taken out of h or rstd as a power of two changes this by less than a factor of two. So with the
call's own rstd, v = h rstd w in 64 bits and |v| below bf16's largest value, y is within E + 2^-8 (|v| + E) + 2^-134 of v,
E = 2 * 2^-24 |v| + 2 * 2^-150 (|w| + 1): half a step of bf16, or half its smallest.
"""

import numpy as np
import pytest
import torch

from oracle import fp8 as o8

from gpu_util import f32, say

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_02_amd import qlora
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return qlora


def check(Y, X, rstd, w):
    h, r, g = (t.double().cpu().numpy() for t in (X, rstd, w))
    got = Y.double().cpu().numpy()
    with np.errstate(all="ignore"):
        v = (h * r[:, None]) * g
        big = 2.0 ** 128 * (1 - 2.0 ** -9)  # from here on bf16 rounds to infinity
        near = np.abs(np.abs(v) - big) <= 2.0 ** -20 * big
        E = 2 * 2.0 ** -24 * np.abs(v) + 2 * 2.0 ** -150 * (np.abs(g) + 1)
        inside = np.abs(got - v) <= E + 2.0 ** -8 * (np.abs(v) + E) + 2.0 ** -134
        good = np.where(np.isnan(v), np.isnan(got), np.where(np.abs(v) >= big, got == np.copysign(np.inf, v), inside))
    assert not near.any()
    bad = np.argwhere(~good)
    say(f"  {len(bad)} of {good.size} outside" + "".join(
        f"; [{m}, {c}] h {h[m, c]:.4g} rstd {r[m]:.4g} w {g[c]:.4g}: {got[m, c]:.6g}, not {v[m, c]:.6g}" for m, c in bad[:4]))
    assert not len(bad)


@pytest.mark.parametrize("k", [8, 63, 128, 192, 1024, 1027, 4096, 8192, 12288, 28672, 32768, 40000, 40001])
@pytest.mark.parametrize("w32", [False, True])
def test_rows_and_gains_at_the_ends_of_the_range(q, k, w32):
    """Finite rows whose squares overflow (rstd 0: y is 0), vanish (rstd infinite where eps is 0) or do neither, with
    gains that take h itself out of fp32's range."""
    g = torch.Generator().manual_seed(k)
    sizes = torch.tensor([3e38, 1e25, 1e18, 1.0, 1e-10, 1e-18, 1e-30, 1e-38])
    X = (torch.rand((8, k), generator=g) * 0.5 + 0.5) * sizes[:, None]
    X = (X * (torch.randint(0, 2, (8, k), generator=g) * 2 - 1)).to(BF).cuda()
    gains = torch.tensor([1.0, 2.0, 1e20, 1e30, 1e-12, 1e-25, 1e-35, 0.0, 0.5])
    w = (gains[torch.arange(k) % 9] * (torch.rand(k, generator=g) * 0.5 + 0.75)).to(F32 if w32 else BF).cuda()
    for eps in (0.0, 1e-5):
        say(f"case: range k={k} w32={w32} eps={eps}")
        Y, _, rstd, x8 = q.rms_norm_fwd(X, w, eps, want_x8=k % 64 == 0)
        assert rstd[0] == 0 and (eps > 0 or torch.isinf(rstd[6]))
        check(Y, X, rstd, w)
        assert (Y[0] == 0).all()
        if x8 is not None:
            codes, scale = o8.encode_rows(f32(Y[:4]))
            assert np.array_equal(x8.codes[:4].cpu().numpy(), codes) and np.array_equal(x8.scale[:4].cpu().numpy(), scale)


@pytest.mark.parametrize("k", [64, 1027, 28672])
def test_zero_and_infinite_factors(q, k):
    """Zeros, infinities and NaN in h and w meet rstd of 0, infinity and NaN as (h rstd) w does, with either gain."""
    X = torch.ones((5, k), dtype=BF)
    X[0], X[1], X[2], X[3, 1], X[4, 1] = 0, 3e38, 1e-30, float("inf"), float("nan")
    X[1, 2], X[2, 2] = 0, 0
    w = torch.ones(k)
    w[3], w[4], w[5], w[6], w[7] = 0, float("inf"), float("nan"), -2, float("-inf")
    for w32 in (False, True):
        Y, _, rstd, _ = q.rms_norm_fwd(X.cuda(), w.to(F32 if w32 else BF).cuda(), 0.0)
        r = rstd.cpu()
        assert torch.isinf(r[0]) and r[1] == 0 and torch.isinf(r[2]) and r[3] == 0 and torch.isnan(r[4])
        want = ((X.float() * r[:, None]) * w).to(BF)
        assert torch.equal(torch.isnan(Y.cpu()), torch.isnan(want))
        assert torch.equal(Y.cpu().nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


@pytest.mark.parametrize("k", [8, 63, 100, 192, 1027, 4096, 8192, 12288, 12001, 28672, 40001])
@pytest.mark.parametrize("w32", [False, True])
def test_gradient_of_rows_at_the_ends_of_the_range(q, k, w32):
    """The forward's rstd of 0 (squares that overflow) passes dres on alone; a rstd that is not finite leaves no finite
    dX in its row and changes no other row."""
    g = torch.Generator().manual_seed(k)
    H, dY, dR = ((torch.randn((40, k), generator=g)).to(BF).cuda() for _ in range(3))
    w = (torch.rand(k, generator=g) + 0.5).to(F32 if w32 else BF).cuda()
    plain = H.clone()
    H[3], H[11], H[12], H[20], H[39] = 3e38, 1e-30, 0, float("inf"), float("nan")
    rstd = q.rms_norm_fwd(H, w, 0.0)[2]
    rstd0 = q.rms_norm_fwd(plain, w, 0.0)[2]
    assert rstd[3] == 0 and torch.isinf(rstd[11]) and torch.isinf(rstd[12]) and rstd[20] == 0 and torch.isnan(rstd[39])
    rest = torch.ones(40, dtype=torch.bool, device="cuda")
    rest[[3, 11, 12, 20, 39]] = False
    for need_dw in (False, True):
        dX = q.rms_norm_bwd(dY, H, rstd, w, dres=dR, need_dw=need_dw)[0]
        want = q.rms_norm_bwd(dY, plain, rstd0, w, dres=dR, need_dw=need_dw)[0]
        assert torch.equal(dX[rest], want[rest])
        assert torch.equal(dX[3], dR[3])
        assert not torch.isfinite(dX[[11, 12, 20, 39]]).any()
