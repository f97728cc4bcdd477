"""Launches of the feed-forward GEMMs that hold whole tiles and tiles split over the contraction at once (more than
256 tiles of 256 x 256, at most 128 of them left over, 16 steps or more), with ragged last rows, columns and steps:
three rows of every row tile, all columns, against the fp64 oracle."""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_02_amd import synth
from oracle import fp8 as o8
from oracle import linear as olin

from gpu_util import check_elementwise, f32, say, sum8_error
from test_gpu_gated import _block, _check_bwd, _check_fwd

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
M = 4300   # 17 row tiles, 17 column tiles below: 256 whole, 33 split in two


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_02_amd import qlora
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return qlora


def _f64(t):
    return t.detach().double().cpu().numpy()


def _normal(shape, std, dt, *seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(synth.rng(*seed).integers(1 << 31)))
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)


def _rows():
    r = sorted({min(256 * t + o, M - 1) for t in range(17) for o in (0, 131, 255)})
    return torch.tensor(r, device="cuda")


@pytest.mark.parametrize("dt", [BF, HF])
def test_fp8_forward_and_dx(q, dt):
    s, r, rows = 0.5, 12, _rows()
    for n, k in ((4200, 2112), (2100, 4160)):          # 17 steps forward (half a block), 17 steps of dX (52 columns of one)
        say(f"case: fp8 tails {n}x{k} {dt}")
        w = q.quantize_fp8(_normal((n, k), 0.02, torch.float32, 80, n))
        X, dY = _normal((M, k), 1.0, dt, 80, n, 1), _normal((M, n), 1.0, dt, 80, n, 2)
        A, B = _normal((r, k), k ** -0.5, dt, 80, n, 3), _normal((n, r), 0.05, dt, 80, n, 4)
        W8 = o8.weight_values(w.codes.cpu().numpy(), w.scale.cpu().numpy(), n, k)
        Ao, Bo, Xo, dYo = _f64(A), _f64(B), _f64(X[rows]), _f64(dY[rows])
        kind = "fp16" if dt == HF else "bf16"
        if n > 4096:
            got, P, Q = q.fp8_linear_fwd(w, X, A, B, s)[0], Xo, W8.T
            ref, lo = o8.linear_fwd(Xo, W8, Ao, Bo, s)[0], (np.abs(Xo) @ np.abs(Ao).T) @ np.abs(Bo).T
        else:
            got, P, Q = q.fp8_linear_bwd(w, None, None, dY, A, B, s, need_dA=False, need_dB=False)[0], dYo, W8
            ref, lo = o8.linear_bwd(Xo, W8, Ao, Bo, s, dYo)[0], (np.abs(dYo) @ np.abs(Bo)) @ np.abs(Ao)
        P8 = np.abs(o8.rows_values(*o8.encode_rows(P), P.shape[1]))
        b = olin._bound(ref, P8 @ np.abs(Q), lo, s, P.shape[1], kind, 256) + sum8_error(P8, Q)
        assert check_elementwise("Y" if n > 4096 else "dX", f32(got[rows]), ref, b) == 0


@pytest.mark.parametrize("dt", [BF, HF])
def test_gated_forward(q, dt):
    n, k, s, rows = 2100, 1088, 0.5, _rows()           # 17 steps and one of the low-rank columns
    say(f"case: gated forward tails {n}x{k} {dt}")
    block = _block(q, n, k, 12, dt)
    X = _normal((M, k), 1.0, dt, 81)
    H, G, U, T = q.gated_fwd(*block[:2], X, *block[2:], s)
    _check_fwd(q, block, X[rows], s, (H[rows], G[rows], U[rows], T[:, rows].contiguous()), dt)


@pytest.mark.parametrize("dt", [BF, HF])
def test_gated_dx(q, dt):
    n, k, s, rows = 520, 4160, 0.5, _rows()            # 18 steps of dG and dU, one of the low-rank columns
    say(f"case: gated dX tails {n}x{k} {dt}")
    block = _block(q, n, k, 12, dt)
    X, dH = _normal((M, k), 1.0, dt, 82, 0), _normal((M, n), 1.0, dt, 82, 1)
    G, U = _normal((M, n), 1.0, dt, 82, 2), _normal((M, n), 1.0, dt, 82, 3)
    dX = q.gated_bwd(*block[:2], None, None, G, U, dH, *block[2:], s, need_dA=False, need_dB=False)[0]
    g, u, d, x = (t[rows].contiguous() for t in (G, U, dH, X))
    part = q.gated_bwd(*block[:2], x, None, g, u, d, *block[2:], s)
    _check_bwd(q, block, x, g, u, d, s, (dX[rows], *part[1:]), dt)
