"""GPU parity of the gated feed-forward block (qlora_gated_fwd / _bwd) against
the fp64 oracle over the same expanded weights: every element of H, G, U and
dX within the bound its arithmetic gives, T and the adapter gradients to 1e-5.
"""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_02_amd import synth
from oracle import fp8 as o8
from oracle import linear as olin
from oracle import mlp as omlp

from gpu_util import GTOL, assert_grad, check_elementwise, f32, report, say

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_02_amd import qlora
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return qlora


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _normal(shape, std, dt, *seed):
    return torch.from_numpy(synth.rng(*seed).standard_normal(shape) * std).to(dt).cuda()


def _block(q, n, k, r, dt, seed=0, std=0.03, **form):
    """(w_gate, w_up, Ag, Bg, Au, Bu)"""
    ws = [q.quantize_nf4(_normal((n, k), std, BF, 41, n, k, seed, i), **form) for i in range(2)]
    if r == 0:
        return (*ws, None, None, None, None)
    lr = [_normal((r, k), k ** -0.5, dt, 41, n, k, seed, 2 + i) for i in range(2)]
    bs = [_normal((n, r), 0.05, dt, 41, n, k, seed, 4 + i) for i in range(2)]
    return (*ws, lr[0], bs[0], lr[1], bs[1])


def _half(dt):
    """Half a step of the type, and of its subnormals."""
    return (2.0 ** -11, 2.0 ** -25) if dt == HF else (2.0 ** -8, 2.0 ** -134)


def _check_fwd(q, block, X, s, out, dt):
    H, G, U, T = out
    wg, wu, Ag, Bg, Au, Bu = block
    Xo = _f64(X)
    Wg, Wu = (_f64(q.dequant(w, dtype=dt)) for w in (wg, wu))
    Hr, Gr, Ur, Tg, Tu = omlp.gated_fwd(Xo, Wg, Wu, *(_f64(t) for t in (Ag, Bg, Au, Bu)), s)
    kind, (u, a) = ("fp16" if dt == HF else "bf16"), _half(dt)
    E = {}
    for name, ref, W, A, B, got in (("G", Gr, Wg, Ag, Bg, G), ("U", Ur, Wu, Au, Bu, U)):
        b = olin.fwd_error_bound(Xo, W, _f64(A), _f64(B), s, ref, out=kind)
        E[name] = (b - a - u * np.abs(ref)) / (1 + u)     # the fp32 sum's own part
        if got is not None:
            assert check_elementwise(name, f32(got), ref, b) == 0
    # H: errors of G and U through silu(G) U (|silu'| <= 1.1), a few fp32 operations, one rounding
    si = np.abs(Gr * omlp.sigmoid(Gr))
    e = 1.1 * E["G"] * (np.abs(Ur) + E["U"]) + si * E["U"] + 2.0 ** -20 * np.abs(Hr)
    assert check_elementwise("H", f32(H), Hr, e + u * (np.abs(Hr) + e) + a) == 0
    assert report("H", f32(H), Hr) <= u
    if T is not None:
        assert_grad("T", T, np.stack([Tg, Tu]))


def _check_bwd(q, block, X, G, U, dH, s, out, dt):
    wg, wu, Ag, Bg, Au, Bu = block
    dX, dAg, dBg, dAu, dBu = out
    Wg, Wu = (_f64(q.dequant(w, dtype=dt)) for w in (wg, wu))
    lr = [_f64(t) for t in (Ag, Bg, Au, Bu)]
    Go, Uo, dHo = _f64(G), _f64(U), _f64(dH)
    ref = omlp.gated_bwd(_f64(X), Wg, Wu, Go, Uo, dHo, *lr, s)
    dG, dU = (np.abs(t) for t in omlp.silu_mul_bwd(Go, Uo, dHo))
    aG, aU = np.abs(Wg), np.abs(Wu)
    u, a = _half(dt)
    # dG, dU: a few fp32 operations (the factor of dG cancels near its zero), then one rounding to 16 bits
    eG = 2.0 ** -20 * np.abs(dHo * Uo) * (1 + np.abs(Go))
    eU = 2.0 ** -20 * dU
    S = dG @ aG + dU @ aU
    E = (eG + u * dG + a) @ aG + (eU + u * dU + a) @ aU
    if Ag is not None:
        L = (dG @ np.abs(lr[1])) @ np.abs(lr[0]) + (dU @ np.abs(lr[3])) @ np.abs(lr[2])
        E = E + (2.0 ** -17 + 2.0 ** -20) * abs(s) * L
        S = S + abs(s) * L
    E = E + olin._gamma(2 * G.shape[1] + 256) * S
    assert check_elementwise("dX", f32(dX), ref[0], E + u * (np.abs(ref[0]) + E) + a) == 0
    assert report("dX", f32(dX), ref[0]) <= 2 * u     # two roundings of half a step each
    if Ag is not None:
        for name, got, want in zip(("dAg", "dBg", "dAu", "dBu"), out[1:], ref[1:]):
            assert_grad(name, got, want)
    else:
        assert out[1:] == (None,) * 4


def _run(q, m, n, k, r, dt, s=0.5, **form):
    block = _block(q, n, k, r, dt, **form)
    X, dH = _normal((m, k), 1.0, dt, 42, m, n, k, 0), _normal((m, n), 1.0, dt, 42, m, n, k, 1)
    out = q.gated_fwd(block[0], block[1], X, *block[2:], s)
    _check_fwd(q, block, X, s, out, dt)
    H, G, U, T = out
    alone = q.gated_fwd(block[0], block[1], X, *block[2:], s, save=False)
    assert torch.equal(alone[0], H) and alone[1:] == (None, None, None)
    back = q.gated_bwd(block[0], block[1], X, T, G, U, dH, *block[2:], s)
    _check_bwd(q, block, X, G, U, dH, s, back, dt)


@pytest.mark.parametrize("m,n,k,r,dt", [
    (1, 64, 64, 1, BF), (1, 1, 128, 0, BF), (16, 1030, 1088, 12, HF), (5, 4200, 192, 0, BF), (16, 8200, 320, 16, BF),
    (3, 8192, 576, 128, HF), (17, 130, 320, 4, BF), (40, 1, 64, 2, BF), (300, 1030, 1088, 12, HF), (257, 100, 640, 5, BF),
    (640, 256, 512, 64, BF), (256, 128, 256, 128, HF), (130, 520, 2048, 16, BF), (33, 31, 4096, 32, BF),
    (520, 2080, 192, 8, BF), (2100, 96, 128, 17, BF),
])
def test_block_against_oracle(q, m, n, k, r, dt):
    say(f"case: gated M={m} N={n} K={k} r={r} {dt}")
    _run(q, m, n, k, r, dt)


@pytest.mark.parametrize("form", [dict(double_quant=False), dict(double_quant=False, scale_dtype=BF)])
@pytest.mark.parametrize("m", [4, 50])
def test_storage_forms(q, m, form):
    say(f"case: gated M={m} {form}")
    _run(q, m, 200, 320, 8, BF, **form)


@pytest.mark.parametrize("m,n,k,r,dt,form", [
    (1, 12307, 512, 7, BF, {}), (16, 4101, 2304, 66, HF, {}), (5, 8209, 256, 128, BF, dict(double_quant=False)),
    (2, 4100, 4864, 12, BF, dict(double_quant=False, scale_dtype=BF)),
    (8, 4130, 2112, 33, BF, dict(double_quant=False, scale_dtype=BF)), (4, 4112, 2304, 0, HF, {}),
])
def test_few_tokens_several_row_groups(q, m, n, k, r, dt, form):
    """More than 256 groups of 16 rows (a workgroup takes several), the last one short, with whole and cut
    256-column chunks, chunk counts that leave waves without one, ranks of every remainder."""
    say(f"case: gated M={m} N={n} K={k} r={r} {dt} {form}")
    _run(q, m, n, k, r, dt, **form)


@pytest.mark.parametrize("m", [2, 16])
def test_levels_of_each_weight_whole_chunks(q, m):
    n, k, s = 4120, 512, 0.5
    grid = torch.tensor(q.build_uniform4_codebook(), device="cuda")
    wg = q.quantize_nf4(_normal((n, k), 0.03, BF, 44, 0))
    wu = q.quantize_nf4(_normal((n, k), 0.03, BF, 44, 1), codebook=grid)
    block = (wg, wu, None, None, None, None)
    X = _normal((m, k), 1.0, BF, 44, 2)
    _check_fwd(q, block, X, s, q.gated_fwd(*block[:2], X, *block[2:], s), BF)


@pytest.mark.parametrize("m,n", [(4, 200), (16, 8200), (50, 200)])
def test_levels_of_each_weight(q, m, n):
    """Gate in NF4, up on the uniform grid: each tile is expanded with its own levels."""
    k, s = 320, 0.5
    grid = torch.tensor(q.build_uniform4_codebook(), device="cuda")
    wg = q.quantize_nf4(_normal((n, k), 0.03, BF, 43, 0))
    wu = q.quantize_nf4(_normal((n, k), 0.03, BF, 43, 1), codebook=grid)
    block = (wg, wu, None, None, None, None)
    X = _normal((m, k), 1.0, BF, 43, 2)
    _check_fwd(q, block, X, s, q.gated_fwd(*block[:2], X, *block[2:], s), BF)


@pytest.mark.parametrize("dt", [BF, HF])
def test_adapter_gradients_hold_fp32(q, dt):
    """The adapter gradients keep the unrounded dG and dU: 24 bits (22 in fp16)
    of each and of T and P, a few fp32 operations each and sums over at most
    1088 terms, so an element misses by a few 2^-22 of its terms, and one lost
    low part (2^-12 of one dG, 5e-6 of the norm here) shows."""
    m, n, k, r, s = 300, 1030, 1088, 12, 0.5
    b = _block(q, n, k, r, dt, seed=5)
    X = _normal((m, k), 1.0, dt, 50, 0)
    G, U, dH = (_normal((m, n), 1.0, dt, 50, 1 + i) for i in range(3))
    T = torch.stack([X.float() @ b[2].float().T, X.float() @ b[4].float().T])
    out = q.gated_bwd(*b[:2], X, T, G, U, dH, *b[2:], s, need_dX=False)
    W = np.zeros((n, k))
    ref = omlp.gated_bwd(_f64(X), W, W, _f64(G), _f64(U), _f64(dH), *(_f64(t) for t in b[2:]), s)
    for name, got, want in zip(("dAg", "dBg", "dAu", "dBu"), out[1:], ref[1:]):
        assert report(name, f32(got), want, floor=False) <= 2.0 ** -20


def test_streamed_activations(q):
    """Activations above 128 MB (the mirrored buffer rotation), forward and dX,
    against fp32 on the GPU on sampled rows."""
    m, s = 16640, 0.5
    for n, k in ((40, 4160), (2100, 64)):
        wg, wu, Ag, Bg, Au, Bu = block = _block(q, n, k, 8, BF, std=0.02)
        X, dH = _normal((m, k), 1.0, BF, 44, n, 0), _normal((m, n), 1.0, BF, 44, n, 1)
        H, G, U, T = q.gated_fwd(wg, wu, X, Ag, Bg, Au, Bu, s)
        out = q.gated_bwd(wg, wu, X, T, G, U, dH, Ag, Bg, Au, Bu, s, need_dA=False, need_dB=False)
        rows = torch.arange(0, m, 331, device="cuda")
        _check_fwd(q, block, X[rows], s, (H[rows], G[rows], U[rows], T[:, rows].contiguous()), BF)
        part = q.gated_bwd(wg, wu, X[rows], T[:, rows].contiguous(), G[rows], U[rows], dH[rows], Ag, Bg, Au, Bu, s)
        _check_bwd(q, block, X[rows], G[rows], U[rows], dH[rows], s, (out[0][rows], *part[1:]), BF)


def test_saturated_gates(q):
    """Gates far from zero on both sides: silu(-big) = -0, its gradient 0, none of it NaN."""
    m, n, k = 40, 64, 64
    w = q.quantize_nf4(torch.eye(64, device="cuda").to(BF))
    X = _normal((m, k), 1.0, BF, 45)
    X[:, 0], X[:, 1], X[:, 2], X[:, 3] = 1000.0, -1000.0, -3e38, 90.0
    for rows in (16, 40):
        x = X[:rows].contiguous()
        H, G, U, T = q.gated_fwd(w, w, x, None, None, None, None, 1.0)
        g = x.float() @ q.dequant(w).float().T
        h = torch.where(g < -200, torch.zeros_like(g), g * torch.sigmoid(g) * g)
        assert torch.isfinite(H).all() and torch.allclose(H.float(), h, rtol=2.0 ** -8, atol=1e-6)
        dH = torch.ones(rows, n, dtype=BF, device="cuda")
        dX = q.gated_bwd(w, w, x, None, G, U, dH, None, None, None, None, 1.0)[0]
        assert torch.isfinite(dX).all() and not dX[:, 1:3].any()


def test_rows_do_not_touch_each_other(q):
    """A row that is not finite stays in its row, forward and dX."""
    n, k, s = 200, 320, 0.5
    b = _block(q, n, k, 8, BF)
    for m in (8, 48):
        X, dH = _normal((m, k), 1.0, BF, 46, m, 0), _normal((m, n), 1.0, BF, 46, m, 1)
        H, G, U, T = q.gated_fwd(*b[:2], X, *b[2:], s)
        dX = q.gated_bwd(*b[:2], X, T, G, U, dH, *b[2:], s)[0]
        X2, G2 = X.clone(), G.clone()
        X2[3, 7] = float("inf")
        G2[3, 9] = float("nan")
        H2 = q.gated_fwd(*b[:2], X2, *b[2:], s)[0]
        dX2 = q.gated_bwd(*b[:2], X, T, G2, U, dH, *b[2:], s, need_dA=False, need_dB=False)[0]
        keep = torch.arange(m, device="cuda") != 3
        assert torch.equal(H2[keep], H[keep]) and torch.equal(dX2[keep], dX[keep])
        assert not torch.isfinite(H2[3]).all() and torch.isnan(dX2[3]).all()


def test_partial_outputs_accumulate_and_empty_batch(q):
    m, n, k, r, s = 48, 200, 320, 8, 0.5
    b = _block(q, n, k, r, BF)
    X, dH = _normal((m, k), 1.0, BF, 47, 0), _normal((m, n), 1.0, BF, 47, 1)
    H, G, U, T = q.gated_fwd(*b[:2], X, *b[2:], s)
    full = q.gated_bwd(*b[:2], X, T, G, U, dH, *b[2:], s)
    assert all(torch.equal(x, y) for x, y in zip(full, q.gated_bwd(*b[:2], X, T, G, U, dH, *b[2:], s)))
    only = q.gated_bwd(*b[:2], None, None, G, U, dH, *b[2:], s, need_dA=False, need_dB=False)
    assert torch.equal(only[0], full[0]) and only[1:] == (None,) * 4
    a = q.gated_bwd(*b[:2], X, T, G, U, dH, *b[2:], s, need_dX=False, need_dB=False)
    assert a[0] is None and torch.equal(a[1], full[1]) and torch.equal(a[3], full[3]) and a[2] is None
    bb = q.gated_bwd(*b[:2], X, None, G, U, dH, *b[2:], s, need_dX=False, need_dA=False)
    assert all(torch.allclose(bb[i], full[i], rtol=0, atol=float(full[i].abs().max()) * GTOL) for i in (2, 4))
    names = ("dA_gate", "dB_gate", "dA_up", "dB_up")
    acc = q.gated_bwd(*b[:2], X, T, G, U, dH, *b[2:], s, accumulate=True, need_dX=False,
                      **{x: t.clone() for x, t in zip(names, full[1:])})
    assert all(torch.equal(x, y + y) for x, y in zip(acc[1:], full[1:]))
    e = q.gated_fwd(*b[:2], X[:0], *b[2:], s)
    assert e[0].shape == (0, n)
    z = q.gated_bwd(*b[:2], X[:0], None, G[:0], U[:0], dH[:0], *b[2:], s)
    assert z[0].shape == (0, k) and not any(t.any() for t in z[1:])


# ------------------------------------------------------- a block of both operators

def _mlp(q, m, d, ff, r, dt, seed):
    b = _block(q, ff, d, r, dt, seed)
    down = q.quantize_fp8(_normal((d, ff), 0.03, torch.float32, 48, seed, 0))
    A, B = _normal((r, ff), ff ** -0.5, dt, 48, seed, 1), _normal((d, r), 0.05, dt, 48, seed, 2)
    X, dY = _normal((m, d), 1.0, dt, 48, seed, 3), _normal((m, d), 1.0, dt, 48, seed, 4)
    return b, down, A, B, X, dY


def _step(q, b, down, A, B, X, dY, s=0.5):
    """Forward and backward of down(silu(gate(x)) * up(x)): gate and up in NF4, down in 8 bits."""
    H, G, U, T = q.gated_fwd(*b[:2], X, *b[2:], s)
    Y, Td = q.fp8_linear_fwd(down, H, A, B, s)
    dH, dA, dB = q.fp8_linear_bwd(down, H, Td, dY, A, B, s)
    return (Y, dA, dB, H, G, U, dH, *q.gated_bwd(*b[:2], X, T, G, U, dH, *b[2:], s))


@pytest.mark.parametrize("m,dt", [(7, BF), (96, HF), (300, BF)])
def test_feed_forward_block_end_to_end(q, m, dt):
    say(f"case: block M={m} {dt}")
    b, down, A, B, X, dY = _mlp(q, m, 256, 704, 8, dt, m)
    Y, dA, dB, H, G, U, dH, *grads = _step(q, b, down, A, B, X, dY)
    W8 = o8.weight_values(down.codes.cpu().numpy(), down.scale.cpu().numpy(), 256, 704)
    _check_fwd(q, b, X, 0.5, (H, G, U, None), dt)
    Yr, _ = o8.linear_fwd(_f64(H), W8, _f64(A), _f64(B), 0.5)
    dHr, dAr, dBr = o8.linear_bwd(_f64(H), W8, _f64(A), _f64(B), 0.5, _f64(dY))
    u = _half(dt)[0]
    assert report("Y", f32(Y), Yr) <= u and report("dH", f32(dH), dHr) <= u
    assert_grad("dA", dA, dAr)
    assert_grad("dB", dB, dBr)
    _check_bwd(q, b, X, G, U, dH, 0.5, grads, dt)


def test_capture_and_replay(q):
    """A captured step of the block, replayed on new inputs with eager work in
    between, equals the eager step every time."""
    for m in (9, 200):
        b, down, A, B, X, dY = _mlp(q, m, 256, 704, 8, BF, m)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            _step(q, b, down, A, B, X, dY)
        torch.cuda.current_stream().wait_stream(st)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _step(q, b, down, A, B, X, dY)
        for i in range(4):
            X.copy_(_normal((m, 256), 1.0, BF, 49, m, i, 0))
            dY.copy_(_normal((m, 256), 1.0, BF, 49, m, i, 1))
            g.replay()
            torch.cuda.synchronize()
            want = _step(q, b, down, A, B, X, dY)
            assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_other_streams(q):
    """Two steps at once on streams of their own, and with the stream argument."""
    cases = [_mlp(q, 130, 256, 704, 8, BF, i) for i in range(2)]
    want = [_step(q, *c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = _step(q, *cases[i])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))
    b, down, A, B, X, dY = cases[0]
    st = streams[0]
    H, G, U, T = q.gated_fwd(*b[:2], X, *b[2:], 0.5, stream=st)
    Y, _ = q.fp8_linear_fwd(down, H, A, B, 0.5, stream=st)
    st.synchronize()
    assert torch.equal(Y, want[0][0]) and torch.equal(H, want[0][3])
