"""CPU pins of the 8-bit oracle: the format against torch's own E4M3
conversion and brute force, the scale rule against its definition, the layer
against fp64 autograd, and the host checks of the 8-bit C ABI (nothing is
launched)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8


def test_table_is_the_format():
    t = fp8.table()
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref, equal_nan=True)
    assert np.nanmax(t) == 448 and np.isnan(t[[0x7F, 0xFF]]).all()


def test_rounding_is_to_nearest_even():
    pos = fp8.table()[:127]
    mid = (pos[1:] + pos[:-1]) / 2
    v = np.concatenate([pos, mid, np.nextafter(mid, 1e9), np.nextafter(mid, 0)])
    got = fp8.encode_values(np.concatenate([v, -v]))
    ref = torch.from_numpy(np.concatenate([v, -v]).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    exact = np.concatenate([v, -v]) == np.concatenate([v, -v]).astype(np.float32)
    assert np.array_equal(got[exact], ref[exact])
    i = np.arange(126)
    assert np.array_equal(fp8.encode_values(mid), i + (i % 2))           # ties: the even code
    assert np.array_equal(fp8.encode_values(np.nextafter(mid, 1e9)), i + 1)
    assert np.array_equal(fp8.encode_values(np.nextafter(mid, 0)), i)
    assert list(fp8.encode_values([np.inf, -np.inf, 0.0, -0.0])) == [0x7F, 0xFF, 0, 0x80]
    assert fp8.encode_values(np.nan) & 0x7F == 0x7F


@pytest.mark.parametrize("amax,byte", [(448.0, 127), (np.nextafter(448.0, 1e9), 128), (1.75, 119), (1.76, 120),
                                       (1.0, 119), (2.0, 120), (0.0, 127), (3.4e38, 247), (2.0 ** -149, 0)])
def test_scale_byte(amax, byte):
    assert fp8.scale_byte(amax) == byte


def test_blocks_are_independent_and_exact_values_return():
    rng = np.random.default_rng(0)
    vals = fp8.table()[:127][rng.integers(0, 127, (3, 192))] * rng.choice([-1, 1], (3, 192))
    vals[:, 0] = vals[:, 128] = 448.0
    c, b = fp8.encode_rows(vals)
    assert c.shape == (3, 256) and b.shape == (3, 2) and (b == 127).all() and (c[:, 192:] == 0).all()
    assert np.array_equal(fp8.rows_values(c, b, 192), vals)
    odd = vals.copy()
    odd[1, 3] = np.nan
    odd[2, 140] = np.inf
    c2, b2 = fp8.encode_rows(odd)
    keep = np.ones(c.shape, bool)
    keep[1, 3] = keep[2, 140] = False
    assert np.array_equal(c2[keep], c[keep]) and np.array_equal(b2, b)
    W = rng.standard_normal((130, 64))
    cw, bw = fp8.encode_weight(W)
    v = fp8.weight_values(cw, bw, 130, 64)
    assert cw.shape == (130, 128) and bw.shape == (2, 1)
    # half a step of 3 mantissa bits, or half the subnormal step of the tile's scale
    assert (np.abs(v - W) <= np.maximum(np.abs(W) * 2.0 ** -4, 2.0 ** -10 * np.ldexp(1.0, int(bw.max()) - 127))).all()


def test_layer_against_autograd_with_the_rounding_passed_through():
    rng = np.random.default_rng(1)
    M, n, k, r, s = 5, 70, 192, 3, 0.5
    X, dY = rng.standard_normal((M, k)), rng.standard_normal((M, n))
    A, B = rng.standard_normal((r, k)), rng.standard_normal((n, r))
    W8 = fp8.weight_values(*fp8.encode_weight(rng.standard_normal((n, k))), n, k)
    q = lambda x: fp8.rows_values(*fp8.encode_rows(x), x.shape[1])  # noqa: E731
    Y, T = fp8.linear_fwd(X, W8, A, B, s)
    tx, ta, tb = (torch.tensor(t, requires_grad=True) for t in (X, A, B))
    base = tx + (torch.tensor(q(X)) - tx).detach()
    y = base @ torch.tensor(W8).T + s * (tx @ ta.T) @ tb.T
    assert np.allclose(y.detach().numpy(), Y, rtol=1e-12, atol=1e-12)
    y.backward(torch.tensor(dY))
    dX, dA, dB = fp8.linear_bwd(X, W8, A, B, s, dY)
    assert np.allclose(ta.grad.numpy(), dA, rtol=1e-10, atol=1e-10)
    assert np.allclose(tb.grad.numpy(), dB, rtol=1e-10, atol=1e-10)
    # dX differs from autograd's by dY's own encoding alone
    assert np.allclose(dX, tx.grad.numpy() + (q(dY) - dY) @ W8, rtol=1e-10, atol=1e-10)


def test_host_checks_of_the_abi():
    from bit_nf4_quantized_02_amd import qlora as q
    lib, p = q.raw(), ctypes.c_void_p(1 << 24)
    off = ctypes.c_void_p((1 << 24) + 8)
    ok, err = ctypes.byref(q._Weight8(100, 192, 1 << 20, 1 << 21)), -1
    assert q.FP8Weight.empty(100, 192, device="cpu").codes.shape == (100, 256)
    assert lib.qlora_fp8_storage_bytes(100, 192) == 100 * 256 + 2
    assert lib.qlora_fp8_storage_bytes(100, 100) == 0 and lib.qlora_fp8_storage_bytes(0, 64) == 0
    bad = ctypes.byref(q._Weight8(100, 100, 1 << 20, 1 << 21))
    null, mis = ctypes.byref(q._Weight8(100, 192, 1 << 20, None)), ctypes.byref(q._Weight8(100, 192, (1 << 20) + 1, 1 << 21))
    big = ctypes.byref(q._Weight8(1 << 23, 192, 1 << 20, 1 << 21))
    for w, want in ((None, err), (bad, -2), (big, -2), (null, err), (mis, err)):
        assert lib.qlora_quantize_fp8(p, 0, w, None) == want
        assert lib.qlora_dequant_fp8(w, p, None) == want
        assert lib.qlora_fp8_linear_fwd(w, p, 4, 0, p, p, 8, 1.0, p, None, p, 1 << 30, None) == want
        assert lib.qlora_fp8_linear_bwd(w, p, None, p, 4, 0, p, p, 8, 1.0, p, p, p, 0, p, 1 << 30, None) == want
    assert lib.qlora_quantize_fp8(p, 3, ok, None) == err and lib.qlora_quantize_fp8(off, 0, ok, None) == err
    assert lib.qlora_dequant_fp8(ok, None, None) == err

    def fwd(X=p, M=40, dt=0, A=p, B=p, r=8, Y=p, T=None, ws=p, nb=None):
        nb = lib.qlora_fp8_linear_workspace_bytes(40, 100, 192, 8, 0) if nb is None else nb
        return lib.qlora_fp8_linear_fwd(ok, X, M, dt, A, B, r, 1.0, Y, T, ws, nb, None)

    assert fwd(dt=1) == err and fwd(dt=7) == err and fwd(X=None) == err and fwd(Y=off) == err and fwd(T=off) == err
    assert fwd(A=None) == err and fwd(B=off) == err and fwd(r=129) == -2 and fwd(r=-1) == -2 and fwd(M=-1) == -2
    assert fwd(M=(1 << 22) + 1) == -2
    assert fwd(ws=None) == -4 and fwd(ws=off) == -4 and fwd(nb=lib.qlora_fp8_linear_workspace_bytes(40, 100, 192, 8, 0) - 1) == -4
    assert fwd(M=0, X=None, Y=None, ws=None, nb=0) == 0

    def bwd(X=p, T=None, dY=p, M=40, dt=0, A=p, B=p, r=8, dX=p, dA=p, dB=p, acc=0, ws=p, nb=None):
        nb = lib.qlora_fp8_linear_workspace_bytes(40, 100, 192, 8, 1) if nb is None else nb
        return lib.qlora_fp8_linear_bwd(ok, X, T, dY, M, dt, A, B, r, 1.0, dX, dA, dB, acc, ws, nb, None)

    assert bwd(dt=1) == err and bwd(acc=2) == err and bwd(dY=None) == err and bwd(X=None) == err
    assert bwd(dX=off) == err and bwd(dA=off) == err and bwd(dB=off) == err and bwd(T=off) == err and bwd(A=None) == err
    assert bwd(r=129) == -2 and bwd(M=-3) == -2 and bwd(ws=None) == -4
    assert bwd(nb=lib.qlora_fp8_linear_workspace_bytes(40, 100, 192, 8, 1) - 1) == -4
    assert bwd(M=0, acc=1) == 0 and bwd(M=0, r=0, dX=None) == 0
    # operands of 4 GiB are refused (M kp here)
    long = ctypes.byref(q._Weight8(64, 1 << 20, 1 << 20, 1 << 21))
    assert lib.qlora_fp8_linear_fwd(long, p, 4096, 0, p, p, 8, 1.0, p, None, p, 1 << 62, None) == -2
    # and the codes for dX, up to the end of the last tile (np kp + 256 bytes)
    for n in (65536, 65535, 65409):
        wide = ctypes.byref(q._Weight8(n, 65536, 1 << 20, 1 << 21))
        assert lib.qlora_fp8_linear_bwd(wide, None, None, p, 40, 0, p, p, 8, 1.0, p, None, None, 0, p, 1 << 62, None) == -2
    for a in ((0, 100, 192, 8, 0), (4, 100, 100, 8, 0), (4, 100, 192, 129, 0), (4, 100, 192, 8, 2)):
        assert lib.qlora_fp8_linear_workspace_bytes(*a) == 0
    # the binding: CPU tensors, wrong types and shapes
    w8 = q.FP8Weight.empty(100, 192, device="cpu")
    with pytest.raises(ValueError):
        q.fp8_linear_fwd(w8, torch.zeros(4, 192, dtype=torch.bfloat16), None, None, 1.0)
    with pytest.raises(ValueError):
        q.quantize_fp8(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        q.quantize_fp8(torch.zeros(4, 64, dtype=torch.int8))
