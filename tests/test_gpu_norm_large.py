"""The norm's largest launches and buffers (qlora_rms_norm_fwd, qlora_rms_norm_bwd): as many rows as the calls take, at
lengths that give each row 1024 threads, 2^32 in all; and offsets past 32 bits in rows of aligned and unaligned lengths,
for dw too.

Bars as in the norm's other tests: the oracle's bounds, which count the roundings.
"""

import numpy as np
import pytest
import torch

from oracle import norm as onorm

from gpu_util import say

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HALF = (2.0 ** -8, 2.0 ** -134)


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_02_amd import qlora
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return qlora


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.fixture
def room():
    def of(nbytes):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        if torch.cuda.mem_get_info()[0] < nbytes + (4 << 30):
            pytest.skip(f"{nbytes >> 30} GiB of device memory are not free")
    yield of
    torch.cuda.empty_cache()


def rows_of(M, k):
    """Zeros but for rows at the ends and around the middle of the launch; which."""
    rows = torch.tensor([0, 1, M // 2 - 1, M // 2, M // 2 + 1, M - 2, M - 1], device="cuda")
    X = torch.zeros((M, k), dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(k)
    X[rows] = torch.randn((len(rows), k), generator=g, device="cuda").to(BF)
    w = (torch.rand(k, generator=g, device="cuda") + 0.5).to(BF)
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[rows] = False
    return X, w, rows, rest


@pytest.mark.parametrize("k", [16378, 16383])
def test_forward_of_most_rows(q, k, room):
    M = 1 << 22
    room(2 * M * k)
    say(f"case: norm forward M={M} k={k}")
    X, w, rows, rest = rows_of(M, k)
    rstd = q.rms_norm_fwd(X, w, 1e-6, rstd=torch.full((M,), -1.0, device="cuda"), want_y=False)[2]
    _, r = onorm.rms_fwd(f64(X[rows]), f64(w), 1e-6)
    assert np.all(np.abs(f64(rstd[rows]) - r) <= r * onorm.rstd_bound(k))
    r0 = np.float64(np.float32(1e-6)) ** -0.5
    assert bool(((rstd[rest].double() - r0).abs() <= r0 * onorm.rstd_bound(k)).all())


def test_gradient_of_most_rows(q, room):
    M, k = 1 << 22, 16383
    room(4 * M * k)
    say(f"case: norm backward M={M} k={k}")
    X, w, rows, rest = rows_of(M, k)
    rstd = torch.full((M,), 0.75, device="cuda")
    dX = torch.full((M, k), 1.0, dtype=BF, device="cuda")
    q.rms_norm_bwd(X, X, rstd, w, need_dw=False, dX=dX)
    args = (f64(X[rows]), f64(X[rows]), f64(rstd[rows]), f64(w), None)
    dx, _ = onorm.rms_bwd(*args)
    assert np.all(np.abs(f64(dX[rows]) - dx) <= onorm.dx_bound(*args, dx, *HALF))
    dX[rows] = 0
    assert not any(bool((part != 0).any()) for part in dX.split(M // 64))


@pytest.mark.parametrize("M,k", [((1 << 19) + 70, 8256), ((1 << 19) + 200, 8255), (1 << 22, 1027), (1 << 22, 1017),
                                 ((1 << 17) + 99, 32769)])
def test_offsets_past_32_bits_in_both_directions(q, room, M, k):
    """More than 2^32 elements (k = 1017: bytes) in a buffer. dY is zero as far as 32 bits reach, and h behind: there dw
    is a sum of positive terms only, none of which another row has; before it dX is dres."""
    first = (1 << (31 if k == 1017 else 32)) // k + 1
    assert first < M
    room(6 * 2 * M * k + (8 << 30))
    say(f"case: norm past 32 bits M={M} k={k}")
    g = torch.Generator(device="cuda").manual_seed(k)
    X, R = (torch.randn((M, k), generator=g, device="cuda", dtype=BF) for _ in range(2))
    w = (torch.rand(k, generator=g, device="cuda") + 0.5).to(BF)
    Y, H, rstd, _ = q.rms_norm_fwd(X, w, 1e-5, residual=R)
    for part in (slice(0, 3), slice(first - 2, first + 3), slice(M - 30, M)):
        assert torch.equal(H[part], (X[part].float() + R[part].float()).to(BF))
        y, r = onorm.rms_fwd(f64(H[part]), f64(w), 1e-5)
        assert np.all(np.abs(f64(rstd[part]) - r) <= r * onorm.rstd_bound(k))
        assert np.all(np.abs(f64(Y[part]) - y) <= onorm.y_bound(y, k, *HALF))
    del X, Y
    dY = torch.zeros_like(H)
    dY[first:] = H[first:]
    dX, dw = q.rms_norm_bwd(dY, H, rstd, w, dres=R)
    alone, none = q.rms_norm_bwd(dY, H, rstd, w, dres=R, need_dw=False)
    assert none is None
    for part in (slice(first, first + 30), slice(M - 30, M)):
        args = (f64(dY[part]), f64(H[part]), f64(rstd[part]), f64(w), f64(R[part]))
        dx, _ = onorm.rms_bwd(*args)
        for got in (dX, alone):
            assert np.all(np.abs(f64(got[part]) - dx) <= onorm.dx_bound(*args, dx, *HALF))
    step = (1 << 28) // k
    for a in range(0, first, step):
        part = slice(a, min(a + step, first))
        assert torch.equal(dX[part], R[part]) and torch.equal(alone[part], R[part])
    want = torch.zeros(k, dtype=torch.float64, device="cuda")
    for a in range(first, M, step):
        part = slice(a, min(a + step, M))
        want += (H[part].double().square() * rstd[part].double()[:, None]).sum(0)
    # (as the oracle's bound of dw, whose terms' magnitudes are the terms here)
    depth = -(-M // 64) + 64 + 32
    assert bool(((dw.double() - want).abs() <= (depth + 3) * onorm.U * want).all())
