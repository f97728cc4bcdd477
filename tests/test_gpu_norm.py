"""GPU parity of the residual addition with the root-mean-square norm (qlora_rms_norm_fwd / _bwd), its 8-bit output and
the 8-bit layer on encoded activations, against the fp64 oracle.

Bars: h bit for bit (one fp32 addition, one rounding); rstd, y, dx, dw within the oracle's bounds, which count the
roundings of an fp32 evaluation (2^-24 each) and half a step of the 16-bit type (bf16 2^-8, fp16 2^-11 of the value, or
half its smallest step); the 8-bit codes and scales equal the oracle's encoding of the call's own y bit for bit, and the
layer on them equals the layer that encodes y itself bit for bit.
"""

import numpy as np
import pytest
import torch

from oracle import fp8 as o8
from oracle import linear as olin
from oracle import norm as onorm

from gpu_util import GTOL, f32, say, sum8_error

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = {BF: (2.0 ** -8, 2.0 ** -134), F16: (2.0 ** -11, 2.0 ** -25)}


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_02_amd import qlora
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return qlora


def f64(t):
    return t.detach().double().cpu().numpy()


def draw(M, k, dt, seed=0, w32=False, res=True):
    g = torch.Generator().manual_seed(seed + 1000 * M + k)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    X, R = r(M, k), r(M, k) * 3
    R[:, ::53] *= 40
    if M > 2:
        X[1], R[1] = 0, 0  # a row of zeros
        X[2] *= 1e-4
        R[2] *= 1e-4
    w = torch.rand(k, generator=g) + 0.5
    dY, dR = r(M, k), r(M, k)
    c = lambda t, d=dt: t.to(d).cuda()  # noqa: E731
    return c(X), c(R) if res else None, c(w, F32 if w32 else dt), c(dY), c(dR)


def check_forward(q, X, R, w, eps, Y, H, rstd):
    dt = X.dtype
    want = X if R is None else (X.float() + R.float()).to(dt)
    assert torch.equal(H.view(torch.int16), want.view(torch.int16))
    y, r = onorm.rms_fwd(f64(H), f64(w), eps)
    k = X.shape[1]
    if rstd is not None:
        assert np.all(np.abs(f64(rstd) - r) <= r * onorm.rstd_bound(k))
    if Y is not None:
        u, tiny = HALF[dt]
        err = np.abs(f64(Y) - y) / onorm.y_bound(y, k, u, tiny)
        say(f"  y: worst {err.max():.3f} of its bound")
        assert err.max() <= 1


# widths: of every form of the kernels and next to where one ends, odd ones, one column
WIDTHS = [1, 7, 8, 64, 100, 120, 121, 122, 128, 129, 130, 132, 136, 248, 249, 250, 255, 256, 264, 505, 506, 511, 512, 520, 1000, 1018, 1024, 1026, 1027,
          1028, 1032, 2041, 2042, 2048, 2056, 4089, 4090, 4096, 4097, 4100, 4104, 5000, 5001, 8185, 8186, 8191, 8192, 8196, 8200,
          16377, 16384, 16392, 20001, 32761, 32762, 32768]


@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("dt", [BF, F16])
def test_forward_and_backward(q, k, dt):
    for M, res, w32 in ((1, True, False), (5, False, True), (67, True, True)):
        say(f"case: norm M={M} k={k} {dt} res={res} w32={w32}")
        X, R, w, dY, dR = draw(M, k, dt, 1, w32, res)
        Y, H, rstd, x8 = q.rms_norm_fwd(X, w, 1e-5, residual=R)
        assert x8 is None
        check_forward(q, X, R, w, 1e-5, Y, H, rstd)
        dR = dR if res else None
        dX, dw = q.rms_norm_bwd(dY, H, rstd, w, dres=dR)
        args = (f64(dY), f64(H), f64(rstd), f64(w), None if dR is None else f64(dR))
        dx, dwx = onorm.rms_bwd(*args)
        err = np.abs(f64(dX) - dx) / onorm.dx_bound(*args, dx, *HALF[dt])
        errw = np.abs(f64(dw) - dwx) - onorm.dw_bound(*args[:3])
        say(f"  dx: worst {err.max():.3f} of its bound; dw: {int((errw > 0).sum())} outside")
        assert err.max() <= 1 and errw.max() <= 0
        # dX alone, dw alone and added to what is there
        only, none = q.rms_norm_bwd(dY, H, rstd, w, dres=dR, need_dw=False)
        assert none is None
        err = np.abs(f64(only) - dx) / onorm.dx_bound(*args, dx, *HALF[dt])
        assert err.max() <= 1
        none, alone = q.rms_norm_bwd(dY, H, rstd, w, need_dX=False)
        assert none is None and torch.equal(alone, dw)
        q.rms_norm_bwd(dY, H, rstd, w, need_dX=False, dw=alone, accumulate=True)
        assert torch.equal(alone, dw + dw)


@pytest.mark.parametrize("k", [*range(2, 26), *range(98, 106), *range(250, 266), 515, 1021, 2045, 4093, 4101])
def test_every_remainder(q, k):
    """Row ends at every place of a 16-byte run, gains in 16 and 32 bits; an infinite gain reaches its own column only."""
    for dt, w32 in ((BF, True), (BF, False), (F16, True)):
        say(f"case: remainder k={k} {dt} w32={w32}")
        X, R, w, dY, dR = draw(9, k, dt, 5, w32, True)
        Y, H, rstd, _ = q.rms_norm_fwd(X, w, 1e-5, residual=R)
        check_forward(q, X, R, w, 1e-5, Y, H, rstd)
        args = (f64(dY), f64(H), f64(rstd), f64(w), f64(dR))
        dx, dwx = onorm.rms_bwd(*args)
        for need_dw in (False, True):
            dX, dw = q.rms_norm_bwd(dY, H, rstd, w, dres=dR, need_dw=need_dw)
            assert np.all(np.abs(f64(dX) - dx) <= onorm.dx_bound(*args, dx, *HALF[dt]))
        assert np.all(np.abs(f64(dw) - dwx) <= onorm.dw_bound(*args[:3]))
        for c in (0, k - 1):
            wi = w.clone()
            wi[c] = float("inf")
            Yi = q.rms_norm_fwd(X, wi, 1e-5, residual=R)[0]
            keep = torch.arange(k, device="cuda") != c
            assert torch.equal(Yi[:, keep], Y[:, keep])
            assert not torch.isfinite(Yi[:, c]).any()


@pytest.mark.parametrize("dt", [BF, F16])
def test_rows_longer_than_a_workgroup_holds(q, dt):
    for M, k in ((3, 32776), (70, 40001), (2, 100032)):
        say(f"case: long rows M={M} k={k} {dt}")
        X, R, w, dY, dR = draw(M, k, dt, 2)
        x8 = q.FP8Rows.empty(M, k) if k % 64 == 0 else None
        Y, H, rstd, _ = q.rms_norm_fwd(X, w, 1e-6, residual=R, x8=x8)
        check_forward(q, X, R, w, 1e-6, Y, H, rstd)
        if x8 is not None:
            codes, scale = o8.encode_rows(f32(Y))
            assert np.array_equal(x8.codes.cpu().numpy(), codes) and np.array_equal(x8.scale.cpu().numpy(), scale)
        dX, dw = q.rms_norm_bwd(dY, H, rstd, w, dres=dR)
        args = (f64(dY), f64(H), f64(rstd), f64(w), f64(dR))
        dx, dwx = onorm.rms_bwd(*args)
        assert np.all(np.abs(f64(dX) - dx) <= onorm.dx_bound(*args, dx, *HALF[dt]))
        assert np.all(np.abs(f64(dw) - dwx) <= onorm.dw_bound(*args[:3]))


@pytest.mark.parametrize("M,k", [(4097, 128), (1500, 64), (5000, 256), (2500, 1024), (3000, 2048), (700, 4096), (1030, 8192),
                                 (300, 12288), (9000, 100), (9001, 200), (9003, 249), (4500, 129), (4400, 506), (2300, 1022), (1200, 2043),
                                 (1100, 3001), (700, 4099), (600, 5001), (600, 8186), (300, 12001)])
def test_many_rows(q, M, k):
    """More rows than the workgroups of the backward hold at once, the last ones not a whole group."""
    X, R, w, dY, dR = draw(M, k, BF, 3)
    Y, H, rstd, _ = q.rms_norm_fwd(X, w, 1e-5, residual=R)
    check_forward(q, X, R, w, 1e-5, Y, H, rstd)
    dX, dw = q.rms_norm_bwd(dY, H, rstd, w, dres=dR)
    args = (f64(dY), f64(H), f64(rstd), f64(w), f64(dR))
    dx, dwx = onorm.rms_bwd(*args)
    assert np.all(np.abs(f64(dX) - dx) <= onorm.dx_bound(*args, dx, *HALF[BF]))
    assert np.all(np.abs(f64(dw) - dwx) <= onorm.dw_bound(*args[:3]))
    again = q.rms_norm_bwd(dY, H, rstd, w, dres=dR)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dw)


@pytest.mark.parametrize("k", [64, 128, 192, 320, 1024, 1984, 4096, 8192, 11008, 28672])
@pytest.mark.parametrize("dt", [BF, F16])
def test_eight_bit_output(q, k, dt):
    for M in (1, 6, 33):
        say(f"case: norm to 8 bits M={M} k={k} {dt}")
        X, R, w, _, _ = draw(M, k, dt, 4)
        Y, H, rstd, x8 = q.rms_norm_fwd(X, w, 1e-5, residual=R, want_x8=True)
        check_forward(q, X, R, w, 1e-5, Y, H, rstd)
        codes, scale = o8.encode_rows(f32(Y))
        assert np.array_equal(x8.codes.cpu().numpy(), codes) and np.array_equal(x8.scale.cpu().numpy(), scale)
        none, H2, norstd, alone = q.rms_norm_fwd(X, w, 1e-5, residual=R, want_y=False, want_x8=True, save=False)
        assert none is None and norstd is None and torch.equal(H2, H)
        assert torch.equal(alone.codes, x8.codes) and torch.equal(alone.scale, x8.scale)
        v = o8.table()[codes] * np.repeat(np.ldexp(1.0, scale.astype(int) - 127), 128, axis=1)
        for t in (BF, F16):
            want = torch.tensor(v[:, :k]).to(t)  # (a product of a 4-bit value and a power of two: no double rounding)
            assert torch.equal(q.dequant_fp8_rows(x8, dtype=t).cpu(), want)


def test_not_finite_values(q):
    """A NaN or an infinity takes its own row with it, as the formulas do, and no other; in the 8-bit form such values
    are NaN and the others keep the scale that they have without them."""
    for dt in (BF, F16):
        X, R, w, dY, dR = draw(40, 256, dt, 5)
        bad = X.clone()
        bad[3, 7], bad[9, 100], bad[20, 255] = float("nan"), float("inf"), float("-inf")
        Y, H, rstd, x8 = q.rms_norm_fwd(bad, w, 1e-5, residual=R, want_x8=True)
        Y0, H0, rstd0, x0 = q.rms_norm_fwd(X, w, 1e-5, residual=R, want_x8=True)
        keep = torch.ones(40, dtype=torch.bool)
        keep[[3, 9, 20]] = False
        for a, b in ((Y, Y0), (H, H0), (rstd, rstd0), (x8.codes, x0.codes), (x8.scale, x0.scale)):
            assert torch.equal(a[keep.cuda()], b[keep.cuda()])
        assert torch.isnan(Y[3]).all() and torch.isnan(rstd[3])
        for m, c in ((9, 100), (20, 255)):
            assert rstd[m] == 0 and torch.isnan(Y[m, c]) and int(torch.isnan(Y[m]).sum()) == 1
            assert (Y[m][~torch.isnan(Y[m])] == 0).all()
        codes, scale = o8.encode_rows(f32(Y))
        assert np.array_equal(x8.scale.cpu().numpy(), scale)
        nan = np.isnan(f32(Y))
        got = x8.codes.cpu().numpy()
        assert np.all((got[nan] & 0x7F) == 0x7F) and np.array_equal(got[~nan], codes[~nan])
        dYb = dY.clone()
        dYb[11, 3] = float("nan")
        dX, _ = q.rms_norm_bwd(dYb, H0, rstd0, w, dres=dR)
        dX0, _ = q.rms_norm_bwd(dY, H0, rstd0, w, dres=dR)
        rest = torch.arange(40, device="cuda") != 11
        assert torch.isnan(dX[11]).all() and torch.equal(dX[rest], dX0[rest])


def test_padding_of_rows_that_are_not_finite(q):
    """The 8-bit form's columns behind the last are zero also where rstd is NaN or infinite."""
    for k in (64, 192, 576, 1088, 4160, 32832):
        X = torch.ones(3, k, dtype=BF, device="cuda")
        X[1, 5], X[2] = float("nan"), 0
        x8 = q.rms_norm_fwd(X, torch.ones(k, dtype=BF, device="cuda"), 0.0, want_x8=True)[3]
        assert (x8.codes[:, k:] == 0).all() and ((x8.codes[1:, :k] & 0x7F) == 0x7F).all(), k
        assert (x8.codes[0, :k] == x8.codes[0, 0]).all()


def test_rows_of_zeros(q):
    X, w = torch.zeros(3, 128, dtype=BF, device="cuda"), torch.ones(128, dtype=BF, device="cuda")
    Y, H, rstd, x8 = q.rms_norm_fwd(X, w, 1e-6, want_x8=True)
    assert (Y == 0).all() and torch.allclose(rstd, torch.full_like(rstd, 1e3)) and (x8.codes == 0).all() and (x8.scale == 127).all()
    dX, dw = q.rms_norm_bwd(torch.ones_like(X), H, rstd, w)
    assert (dw == 0).all() and torch.equal(dX, torch.full_like(dX, 1000))


def test_in_place_and_outputs_given(q):
    for k in (256, 8192, 33000):
        X, R, w, dY, dR = draw(20, k, BF, 6)
        Y, H, rstd, _ = q.rms_norm_fwd(X, w, 1e-5, residual=R)
        dX, dw = q.rms_norm_bwd(dY, H, rstd, w, dres=dR)
        stream, out = R.clone(), torch.full((20, k), 7.0, dtype=BF, device="cuda")
        r = torch.empty(20, device="cuda")
        Y2, H2, r2, _ = q.rms_norm_fwd(X, w, 1e-5, residual=stream, H=stream, Y=out, rstd=r)
        assert Y2 is out and H2 is stream and r2 is r
        assert torch.equal(stream, H) and torch.equal(out, Y) and torch.equal(r, rstd)
        grad = dR.clone()
        dX2, dw2 = q.rms_norm_bwd(dY, H, rstd, w, dres=grad, dX=grad)
        assert dX2 is grad and torch.equal(grad, dX) and torch.equal(dw2, dw)


def test_rows_behind_the_last_are_left_alone(q):
    """Outputs that are the front of larger buffers: what lies behind stays as it was."""
    for M, k in ((3, 64), (5, 200), (2, 1027), (5, 129), (3, 100), (7, 2050), (3, 4096)):
        X, R, w, dY, dR = draw(M, k, BF, 7)
        big = lambda dt=BF: torch.full((M + 40, k), 5.0, dtype=dt, device="cuda")  # noqa: E731
        by, bh, br, bx = big(), big(), torch.full((M + 64,), 5.0, device="cuda"), big()
        q.rms_norm_fwd(X, w, 1e-5, residual=R, Y=by[:M], H=bh[:M], rstd=br[:M])
        bw = torch.full((k + 64,), 5.0, device="cuda")
        q.rms_norm_bwd(dY, bh[:M], br[:M], w, dres=dR, dX=bx[:M], dw=bw[:k])
        assert all((b[M:] == 5).all() for b in (by, bh, br, bx)) and (bw[k:] == 5).all()
        if k % 64 == 0:
            kb = -(-k // 128)
            codes = torch.full((M + 40, 128 * kb), 9, dtype=torch.uint8, device="cuda")
            scale = torch.full((M + 40, kb), 9, dtype=torch.uint8, device="cuda")
            q.rms_norm_fwd(X, w, 1e-5, residual=R, x8=q.FP8Rows(M, k, codes[:M], scale[:M]))
            assert (codes[M:] == 9).all() and (scale[M:] == 9).all()


def test_empty_batch(q):
    w = torch.ones(64, dtype=BF, device="cuda")
    X = torch.empty(0, 64, dtype=BF, device="cuda")
    Y, H, rstd, x8 = q.rms_norm_fwd(X, w, 1e-5, residual=X, want_x8=True)
    assert Y.shape == (0, 64) and H.shape == (0, 64) and rstd.shape == (0,) and x8.codes.shape == (0, 128)
    dX, dw = q.rms_norm_bwd(X, X, rstd, w, dw=torch.full((64,), 3.0, device="cuda"))
    assert dX.shape == (0, 64) and (dw == 0).all()
    _, dw = q.rms_norm_bwd(X, X, rstd, w, dw=torch.full((64,), 3.0, device="cuda"), accumulate=True)
    assert (dw == 3).all()
    assert q.dequant_fp8_rows(x8).shape == (0, 64)


def test_offsets_past_32_bits(q):
    """More than 2^32 elements in a buffer: the last rows are right, with and without 8-bit output."""
    M, k = (1 << 19) + 70, 8256
    g = torch.Generator(device="cuda").manual_seed(8)
    X = torch.randn((M, k), generator=g, device="cuda", dtype=BF)
    w = (torch.rand(k, generator=g, device="cuda") + 0.5).to(BF)
    Y, H, rstd, x8 = q.rms_norm_fwd(X, w, 1e-5, want_x8=True)
    tail = slice(M - 40, M)
    check_forward(q, X[tail], None, w, 1e-5, Y[tail], H[tail], rstd[tail])
    codes, scale = o8.encode_rows(f32(Y[tail]))
    assert np.array_equal(x8.codes[tail].cpu().numpy(), codes) and np.array_equal(x8.scale[tail].cpu().numpy(), scale)
    back = q.dequant_fp8_rows(x8)
    v = o8.table()[codes] * np.repeat(np.ldexp(1.0, scale.astype(int) - 127), 128, axis=1)
    assert np.array_equal(f32(back[tail]), v[:, :k])
    del back
    dX, dw = q.rms_norm_bwd(Y, X, rstd, w)
    args = (f64(Y[tail]), f64(X[tail]), f64(rstd[tail]), f64(w), None)
    dx, _ = onorm.rms_bwd(*args)
    assert np.all(np.abs(f64(dX[tail]) - dx) <= onorm.dx_bound(*args, dx, *HALF[BF]))


@pytest.mark.parametrize("M", [1, 3, 8, 9, 16, 17, 32, 33, 63, 64, 65, 128, 300])
@pytest.mark.parametrize("n,k,r", [(96, 128, 8), (1030, 1088, 12), (4200, 512, 0), (256, 4096, 64), (77, 192, 128), (50, 64, 3)])
@pytest.mark.parametrize("dt", [BF, F16])
def test_layer_on_encoded_activations(q, M, n, k, r, dt):
    """The layer on the norm's codes: right by the oracle, and bit for bit the layer that encodes the norm's 16-bit
    output, except for the 17 to 64 tokens that take another kernel there."""
    X, R, w, _, _ = draw(M, k, dt, 9)
    g = torch.Generator().manual_seed(n)
    w8 = q.quantize_fp8((torch.randn((n, k), generator=g) * 0.05).to(dt).cuda())
    A = ((torch.rand((r, k), generator=g) * 2 - 1) * k ** -0.5).to(dt).cuda() if r else None
    B = (torch.randn((n, r), generator=g) * 0.05).to(dt).cuda() if r else None
    Y, _, _, x8 = q.rms_norm_fwd(X, w, 1e-5, residual=R, want_x8=True)
    got, T = q.fp8_linear_fwd_rows(w8, x8, Y if r else None, A, B, 0.5, dtype=dt)
    assert (T is None) == (r == 0)
    if M <= 16 or M > 64:
        out, T2 = q.fp8_linear_fwd(w8, Y, A, B, 0.5)
        assert torch.equal(got, out) and (r == 0 or torch.equal(T, T2))
    if M <= 65 and n <= 1030:
        kp = -(-k // 128) * 128
        W = o8.table()[w8.codes.cpu().numpy()]
        W *= np.ldexp(1.0, np.repeat(np.repeat(w8.scale.cpu().numpy().astype(int) - 127, 128, 0)[:n], 128, 1))
        V = o8.table()[x8.codes.cpu().numpy()] * np.repeat(np.ldexp(1.0, x8.scale.cpu().numpy().astype(int) - 127), 128, 1)
        base, S = V @ W.T, np.abs(V) @ np.abs(W).T
        low = 0.5 * (f64(Y) @ f64(A).T) @ f64(B).T if r else 0.0
        Sl = 0.5 * (np.abs(f64(Y)) @ np.abs(f64(A)).T) @ np.abs(f64(B)).T if r else 0.0
        # the 8-bit sums' own error, fp32 sums of kp + 2 r terms and T's, T's pair of 16-bit parts (2^-16), the output
        E = sum8_error(V, W.T) + (kp + r + 300) * 2.0 ** -23 * (S + Sl) + 2.0 ** -16 * Sl
        ref = base + low
        assert np.all(np.abs(f64(got) - ref) <= E + HALF[dt][0] * (np.abs(ref) + E) + HALF[dt][1])
    if r:
        assert olin.relerr(f32(T), f64(Y) @ f64(A).T) <= GTOL


def test_few_tokens_over_weights_of_both_sizes(q):
    """33 to 64 tokens: one pass over the codes for a weight of 64 MB, the GEMM for a larger one; both the product."""
    k = 4096
    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn((50, k), generator=g, device="cuda").to(BF)
    Y, _, _, x8 = q.rms_norm_fwd(X, torch.ones(k, dtype=BF, device="cuda"), 1e-5, want_x8=True)
    V = q.dequant_fp8_rows(x8).double()
    for n in (16384, 16400):
        w8 = q.quantize_fp8(torch.randn((n, k), generator=g, device="cuda") * 0.02)
        got = q.fp8_linear_fwd_rows(w8, x8, None, None, None, 1.0)[0]
        W = q.dequant_fp8(w8).double()
        ref, S = V @ W.T, V.abs() @ W.abs().T
        # a sum of eight loses at most 7 2^-13 of its largest product, which is at most the sum of all eight
        E = (7 * 2.0 ** -13 + (k + 300) * 2.0 ** -23) * S
        assert bool(((got.double() - ref).abs() <= E + 2.0 ** -8 * (ref.abs() + E)).all()), n
        assert float((got.double() - ref).norm() / ref.norm()) <= 2e-3


def test_codes_of_other_rows_do_not_matter(q):
    """Few tokens: operand rows past the last token are not those of anything behind the codes."""
    n, k = 200, 256
    g = torch.Generator().manual_seed(11)
    w8 = q.quantize_fp8((torch.randn((n, k), generator=g) * 0.05).to(BF).cuda())
    codes = torch.full((80, k), 0x7F, dtype=torch.uint8, device="cuda")     # NaN behind the last row
    scale = torch.full((80, k // 128), 255, dtype=torch.uint8, device="cuda")
    for M in (3, 11, 19, 37):
        X, R, w, _, _ = draw(M, k, BF, 12)
        x8 = q.FP8Rows(M, k, codes[:M], scale[:M])
        q.rms_norm_fwd(X, w, 1e-5, residual=R, x8=x8)
        got, _ = q.fp8_linear_fwd_rows(w8, x8, None, None, None, 1.0)
        assert bool(torch.isfinite(got).all())
        for m in (0, M - 1):  # a token's sums do not depend on the others
            one = q.FP8Rows(1, k, codes[m:m + 1].clone(), scale[m:m + 1].clone())
            assert torch.equal(q.fp8_linear_fwd_rows(w8, one, None, None, None, 1.0)[0][0], got[m])


def test_another_stream_and_captured(q):
    """On a stream of its own, and captured and replayed several times with new inputs and eager work between."""
    M, k, n, r = 70, 1088, 300, 8
    X, R, w, dY, dR = draw(M, k, BF, 13)
    g = torch.Generator().manual_seed(3)
    w8 = q.quantize_fp8((torch.randn((n, k), generator=g) * 0.05).to(BF).cuda())
    A, B = (torch.randn((r, k), generator=g) * 0.03).to(BF).cuda(), (torch.randn((n, r), generator=g) * 0.05).to(BF).cuda()

    def step():
        Y, H, rstd, x8 = q.rms_norm_fwd(X, w, 1e-5, residual=R, want_x8=True)
        out, T = q.fp8_linear_fwd_rows(w8, x8, Y, A, B, 0.5)
        dX, dw = q.rms_norm_bwd(dY, H, rstd, w, dres=dR)
        return [Y, H, rstd, x8.codes, x8.scale, out, T, dX, dw, q.dequant_fp8_rows(x8)]

    want = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Y, H, rstd, _ = q.rms_norm_fwd(X, w, 1e-5, residual=R, stream=s)
    dX, dw = q.rms_norm_bwd(dY, H, rstd, w, dres=dR, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip((Y, H, rstd, dX, dw), (want[0], want[1], want[2], want[7], want[8])):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        outs = step()
    for i in range(4):
        X.copy_(torch.randn(M, k, generator=g).to(BF))
        dY.mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b), i


def test_two_calls_at_once(q):
    """Calls that overlap on two streams, with outputs and workspaces of their own."""
    sets = [draw(2000, k, BF, 14) for k in (1024, 1027)]
    want = []
    for X, R, w, dY, dR in sets:
        Y, H, rstd, _ = q.rms_norm_fwd(X, w, 1e-5, residual=R)
        want.append([Y, H, rstd, *q.rms_norm_bwd(dY, H, rstd, w, dres=dR)])
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, (X, R, w, dY, dR) in zip(streams, sets):
            Y, H, rstd, _ = q.rms_norm_fwd(X, w, 1e-5, residual=R, stream=s)
            got.append([Y, H, rstd, *q.rms_norm_bwd(dY, H, rstd, w, dres=dR, stream=s)])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, v in zip(got, want) for a, b in zip(g, v))


def test_two_graphs_with_one_workspace(q):
    """Replayed after one another on a stream, each leaves its own results."""
    sets = [draw(300, k, BF, 15) for k in (512, 4096)]
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    graphs, outs, want, s = [], [], [], torch.cuda.Stream()
    for X, R, w, dY, dR in sets:
        Y, H, rstd, _ = q.rms_norm_fwd(X, w, 1e-5, residual=R)
        want.append(q.rms_norm_bwd(dY, H, rstd, w, dres=dR, ws=ws))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(q.rms_norm_bwd(dY, H, rstd, w, dres=dR, ws=ws))
        graphs.append((g, H, rstd))
    for _ in range(3):
        for g, _, _ in graphs:
            g.replay()
        ws.fill_(255)
        torch.cuda.synchronize()
        for (dX, dw), (a, b) in zip(outs, want):
            assert torch.equal(dX, a) and torch.equal(dw, b)
            dw.zero_()


def test_refusals_on_the_device(q):
    X, R, w, dY, dR = draw(8, 128, BF, 16)
    Y, H, rstd, x8 = q.rms_norm_fwd(X, w, 1e-5, residual=R, want_x8=True)
    w8 = q.quantize_fp8(torch.ones(64, 128, device="cuda"))
    A, B = torch.zeros(4, 128, dtype=BF, device="cuda"), torch.zeros(64, 4, dtype=BF, device="cuda")
    half, other = X[:, ::2], torch.zeros(8, 128, dtype=F16, device="cuda")
    for call in (lambda: q.rms_norm_fwd(half, w[:64], 1e-5), lambda: q.rms_norm_fwd(X.t(), w[:8], 1e-5),
                 lambda: q.rms_norm_fwd(X, w[:64], 1e-5), lambda: q.rms_norm_fwd(X, w.to(F16), 1e-5),
                 lambda: q.rms_norm_fwd(X, w, 1e-5, residual=other), lambda: q.rms_norm_fwd(X, w, 1e-5, H=H),
                 lambda: q.rms_norm_fwd(X, w, 1e-5, Y=Y[:4]), lambda: q.rms_norm_fwd(X, w, 1e-5, rstd=rstd[:4]),
                 lambda: q.rms_norm_fwd(X, w, 1e-5, x8=q.FP8Rows(8, 128, x8.codes[:4], x8.scale)),
                 lambda: q.rms_norm_bwd(dY, H[:4], rstd, w), lambda: q.rms_norm_bwd(dY, H, rstd.double(), w),
                 lambda: q.rms_norm_bwd(dY, H, rstd, w, dres=other), lambda: q.rms_norm_bwd(dY, H, rstd, w, dw=w),
                 lambda: q.rms_norm_bwd(dY, H, rstd, w, ws=torch.empty(1 << 20, dtype=torch.uint8)),
                 lambda: q.fp8_linear_fwd_rows(w8, x8, None, A, B, 1.0), lambda: q.fp8_linear_fwd_rows(w8, x8, other, A, B, 1.0),
                 lambda: q.fp8_linear_fwd_rows(w8, x8, Y, None, B, 1.0),
                 lambda: q.fp8_linear_fwd_rows(w8, q.FP8Rows(8, 128, x8.codes.cpu(), x8.scale), None, None, None, 1.0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: q.rms_norm_fwd(X, w, -1.0), lambda: q.rms_norm_fwd(X, w, float("nan")),
                 lambda: q.rms_norm_fwd(X[:, :100].contiguous(), w[:100], 1e-5, want_x8=True),
                 lambda: q.rms_norm_fwd(X.view(-1)[1:1 + 128].view(1, 128), w, 1e-5),                # not aligned
                 lambda: q.rms_norm_bwd(dY, H, rstd, w, ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
                 lambda: q.fp8_linear_fwd_rows(q.quantize_fp8(torch.ones(64, 192, device="cuda")), x8, None, None, None, 1.0)):
        with pytest.raises(q.QLoraError):
            call()
    assert torch.equal(q.rms_norm_fwd(X, w, 1e-5, residual=R)[0], Y)  # and is still usable
