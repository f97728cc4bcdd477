"""GPU parity of the 8-bit layer (qlora_quantize_fp8, qlora_dequant_fp8,
qlora_fp8_linear_fwd / _bwd) against the fp64 oracle: codes, scales and
decoded values bit for bit; Y and dX within the element-wise bound of an
fp32-accumulated 16-bit result over the same 8-bit values; T, dA, dB to 1e-5.
"""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_02_amd import synth
from oracle import fp8 as o8
from oracle import linear as olin

from gpu_util import assert_grad, bits16, check_elementwise, f32, report, say

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_02_amd import qlora
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return qlora


def _f64(t):
    return t.detach().double().cpu().numpy()


def _normal(shape, std, dt, *seed):
    return torch.from_numpy(synth.rng(*seed).standard_normal(shape) * std).to(dt)


@pytest.mark.parametrize("n,k,dt", [(1, 64, BF), (128, 128, torch.float32), (130, 192, HF), (257, 1088, BF),
                                    (1000, 4096, torch.float32)])
def test_encode_and_decode_bit_for_bit(q, n, k, dt):
    say(f"case: fp8 encode {n}x{k} {dt}")
    W = _normal((n, k), 0.02, dt, 31, n, k)
    W.view(-1)[::97] *= 10
    W[:, : k // 2] *= 2.0 ** -6                       # tiles of different scales
    if n > 128:
        W[128:, :64] = 0
    w = q.quantize_fp8(W.cuda())
    v = q.dequant_fp8(w)
    torch.cuda.synchronize()
    codes, b = o8.encode_weight(W.double().numpy())
    assert np.array_equal(w.scale.cpu().numpy(), b)
    assert np.array_equal(w.codes.cpu().numpy(), codes)
    ref = torch.from_numpy(o8.weight_values(codes, b, n, k)).to(BF)
    assert np.array_equal(bits16(v), bits16(ref))


def test_encode_extremes(q):
    """Zeros, the largest and smallest magnitudes, midpoints between codes,
    values that are not finite."""
    t = o8.table()[:127]
    mid = np.concatenate([(t[1:] + t[:-1]) / 2, t, [448.0]])
    W = np.zeros((640, 128), np.float32)
    W[0, : len(mid[:128])] = mid[:128]
    W[1, : len(mid[128:])] = mid[128:]
    W[128, :4] = [3.4e38, -1e38, 1e30, 1e-38]
    W[256, :4] = [2.0 ** -149, -(2.0 ** -126), 2.0 ** -130, 0]
    W[384, :4] = [np.nan, np.inf, -np.inf, 1.0]
    W[512:] = np.inf
    w = q.quantize_fp8(torch.from_numpy(W).cuda())
    codes, b = o8.encode_weight(W)
    got = w.codes.cpu().numpy()
    nan = (codes & 0x7F) == 0x7F
    assert np.array_equal(w.scale.cpu().numpy(), b)
    assert np.array_equal(got[~nan], codes[~nan]) and ((got[nan] & 0x7F) == 0x7F).all()
    v = q.dequant_fp8(w).float().cpu().numpy()
    assert np.array_equal(np.isnan(v), nan)
    ref = torch.from_numpy(o8.weight_values(codes, b, 640, 128)).to(BF).float().numpy()
    assert np.array_equal(v[~nan], ref[~nan])


def _bound(Zref, main, lora, s, n, dt):
    return olin._bound(Zref, main, lora, s, n, "fp16" if dt == HF else "bf16", 256)


def _check_layer(q, m, n, k, r, dt, s=0.5, xstd=1.0):
    X, dY = _normal((m, k), xstd, dt, 32, m, n, k, 0), _normal((m, n), 1.0, dt, 32, m, n, k, 1)
    A = _normal((r, k), k ** -0.5, dt, 32, m, n, k, 2) if r else None
    B = _normal((n, r), 0.05, dt, 32, m, n, k, 3) if r else None
    w = q.quantize_fp8(_normal((n, k), 0.02, torch.float32, 32, n, k).cuda())
    g = lambda t: None if t is None else t.cuda()  # noqa: E731
    Y, T = q.fp8_linear_fwd(w, g(X), g(A), g(B), s)
    dX, dA, dB = q.fp8_linear_bwd(w, g(X), T, g(dY), g(A), g(B), s)
    torch.cuda.synchronize()
    W8 = o8.weight_values(w.codes.cpu().numpy(), w.scale.cpu().numpy(), n, k)
    Xo, dYo = _f64(X), _f64(dY)
    Ao, Bo = (None, None) if r == 0 else (_f64(A), _f64(B))
    Yr, Tr = o8.linear_fwd(Xo, W8, Ao, Bo, s)
    dXr, dAr, dBr = o8.linear_bwd(Xo, W8, Ao, Bo, s, dYo)
    X8 = np.abs(o8.rows_values(*o8.encode_rows(Xo), k))
    Y8 = np.abs(o8.rows_values(*o8.encode_rows(dYo), n))
    ly = lx = 0.0
    if r:
        ly = (np.abs(Xo) @ np.abs(Ao).T) @ np.abs(Bo).T
        lx = (np.abs(dYo) @ np.abs(Bo)) @ np.abs(Ao)
    assert check_elementwise("Y", f32(Y), Yr, _bound(Yr, X8 @ np.abs(W8).T, ly, s, k, dt)) == 0
    assert check_elementwise("dX", f32(dX), dXr, _bound(dXr, Y8 @ np.abs(W8), lx, s, n, dt)) == 0
    half = 2.0 ** (-11 if dt == HF else -8)  # half a step
    assert report("Y", f32(Y), Yr) <= half and report("dX", f32(dX), dXr) <= half
    if r:
        assert_grad("T", T, Tr)
        assert_grad("dA", dA, dAr)
        assert_grad("dB", dB, dBr)
    else:
        assert T is None and dA is None and dB is None


@pytest.mark.parametrize("m,n,k,r,dt", [
    (1, 64, 64, 1, BF), (1, 8200, 192, 0, HF), (5, 1, 1024, 4, BF), (16, 1000, 2048, 16, BF), (16, 8224, 4160, 128, HF),
    (17, 130, 320, 4, BF), (40, 1030, 1088, 12, HF), (257, 100, 640, 5, BF), (300, 1030, 1088, 12, HF),
    (640, 256, 512, 64, BF), (256, 128, 256, 128, HF), (130, 520, 8320, 16, BF), (2, 300, 4096, 0, BF),
])
def test_layer_against_oracle(q, m, n, k, r, dt):
    say(f"case: fp8 layer M={m} N={n} K={k} r={r} {dt}")
    _check_layer(q, m, n, k, r, dt)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 7, 8, 13])
def test_gemm_step_remainders(q, steps):
    """Every remainder of the buffer rotation, forward and dX."""
    say(f"case: fp8 layer {steps} steps")
    _check_layer(q, 64, 128 * steps, 128 * steps, 8, BF)


def test_scales_far_apart(q):
    """Rows of X at 2^-60 .. 2^60 (bf16): each output row carries its scale exactly."""
    m, n, k = 40, 256, 384
    X = _normal((m, k), 1.0, BF, 33)
    e = torch.linspace(-60, 60, m).round()
    w = q.quantize_fp8(_normal((n, k), 0.02, torch.float32, 34).cuda())
    for rows in (slice(0, 40), slice(0, 16)):      # the GEMM and the GEMV
        Y, _ = q.fp8_linear_fwd(w, X[rows].contiguous().cuda(), None, None, 1.0)
        p = torch.ldexp(torch.ones(m), e.int())[rows, None]
        Z, _ = q.fp8_linear_fwd(w, (X[rows].float() * p).to(BF).cuda(), None, None, 1.0)
        assert torch.equal(Z.cpu(), (Y.cpu().float() * p).to(BF))


def test_values_not_finite_stay_visible(q):
    m, n, k = 40, 256, 384
    X = _normal((m, k), 1.0, BF, 35)
    w = q.quantize_fp8(_normal((n, k), 0.02, torch.float32, 36).cuda())
    bad = X.clone()
    bad[3, 5], bad[7, 300] = float("nan"), float("inf")
    for rows in (slice(0, 40), slice(0, 16)):
        Y, _ = q.fp8_linear_fwd(w, X[rows].contiguous().cuda(), None, None, 1.0)
        Z, _ = q.fp8_linear_fwd(w, bad[rows].contiguous().cuda(), None, None, 1.0)
        hit = torch.zeros(Z.shape[0], dtype=torch.bool)
        hit[[3, 7]] = True
        assert torch.isnan(Z[hit.cuda()]).all() and torch.equal(Z[~hit.cuda()], Y[~hit.cuda()])


def test_empty_batch_accumulate_and_partial_outputs(q):
    m, n, k, r, s = 48, 200, 320, 8, 0.5
    X, dY = _normal((m, k), 1.0, BF, 37, 0).cuda(), _normal((m, n), 1.0, BF, 37, 1).cuda()
    A, B = _normal((r, k), 0.05, BF, 37, 2).cuda(), _normal((n, r), 0.05, BF, 37, 3).cuda()
    w = q.quantize_fp8(_normal((n, k), 0.02, BF, 37, 4).cuda())
    Y, T = q.fp8_linear_fwd(w, X, A, B, s)
    dX, dA, dB = q.fp8_linear_bwd(w, X, T, dY, A, B, s)
    d2 = q.fp8_linear_bwd(w, X, None, dY, A, B, s, need_dX=False)
    assert d2[0] is None and torch.equal(d2[1], dA) and torch.allclose(d2[2], dB, rtol=0, atol=1e-5)
    d3 = q.fp8_linear_bwd(w, None, None, dY, A, B, s, need_dA=False, need_dB=False)
    assert torch.equal(d3[0], dX) and d3[1] is None and d3[2] is None
    acc = q.fp8_linear_bwd(w, X, T, dY, A, B, s, dA=dA.clone(), dB=dB.clone(), accumulate=True)
    assert torch.equal(acc[1], dA + dA) and torch.equal(acc[2], dB + dB)
    e = q.fp8_linear_fwd(w, X[:0], A, B, s)
    assert e[0].shape == (0, n)
    z = q.fp8_linear_bwd(w, X[:0], None, dY[:0], A, B, s)
    assert not z[1].any() and not z[2].any() and z[0].shape == (0, k)
    again = q.fp8_linear_bwd(w, X, T, dY, A, B, s)
    assert all(torch.equal(a, b) for a, b in zip(again, (dX, dA, dB)))


@pytest.mark.parametrize("n,k,r", [(1030, 1088, 8), (70, 320, 0), (8192 + 9, 192, 4)])
def test_bytes_around_the_weight_are_not_read_as_codes(q, n, k, r):
    """The same weight inside a buffer whose other bytes are NaN codes gives the same results: the tiles of
    the forward, of dX (whose contraction ends inside one) and of the single-token form end with the weight."""
    w = q.quantize_fp8(_normal((n, k), 0.02, torch.float32, 38, n, k).cuda())
    buf = torch.full((n + 512, w.codes.shape[1]), 0x7F, dtype=torch.uint8, device="cuda")
    buf[256:256 + n] = w.codes
    inner = q.FP8Weight(n, k, buf[256:256 + n], w.scale)
    A = _normal((r, k), 0.05, BF, 38, 1).cuda() if r else None
    B = _normal((n, r), 0.05, BF, 38, 2).cuda() if r else None
    for m in (1, 16, 40, 300):
        say(f"case: fp8 inside NaN codes M={m} N={n} K={k}")
        X, dY = _normal((m, k), 1.0, BF, 38, m, 3).cuda(), _normal((m, n), 1.0, BF, 38, m, 4).cuda()
        a, b = (q.fp8_linear_fwd(v, X, A, B, 0.5) for v in (w, inner))
        assert torch.isfinite(a[0]).all() and torch.equal(a[0], b[0])
        a, b = (q.fp8_linear_bwd(v, X, None, dY, A, B, 0.5) for v in (w, inner))
        assert torch.isfinite(a[0]).all() and torch.equal(a[0], b[0])


def test_binding_refuses_what_the_call_does_not_take(q):
    m, n, k, r = 20, 64, 128, 4
    w = q.quantize_fp8(_normal((n, k), 0.02, BF, 39, 0).cuda())
    X, dY = _normal((m, k), 1.0, BF, 39, 1).cuda(), _normal((m, n), 1.0, BF, 39, 2).cuda()
    A, B = _normal((r, k), 0.05, BF, 39, 3).cuda(), _normal((n, r), 0.05, BF, 39, 4).cuda()
    for a, b in ((A, None), (A, B.cpu()), (A, B.half()), (A, B.t()), (A[:, :64], B), (A.t(), B)):
        with pytest.raises(ValueError):
            q.fp8_linear_fwd(w, X, a, b, 0.5)
        with pytest.raises(ValueError):
            q.fp8_linear_bwd(w, X, None, dY, a, b, 0.5)
    for x, y in ((X.half(), dY), (X[:, :64], dY), (X, dY[:, :32]), (X[:3], dY)):
        with pytest.raises(ValueError):
            q.fp8_linear_bwd(w, x, None, y, A, B, 0.5)
    with pytest.raises(ValueError):
        q.fp8_linear_bwd(w, X, torch.zeros(m, r + 1, device="cuda"), dY, A, B, 0.5)
    with pytest.raises(ValueError):
        q.fp8_linear_fwd(w, X, A, B, 0.5, Y=torch.empty(m, n, device="cuda"))
