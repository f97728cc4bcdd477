"""The binding of the feed-forward operators refuses half an adapter, whichever half is missing: a B without its A
would otherwise leave the call without the adapter that its caller passed."""

import pytest
import torch

from bit_nf4_quantized_02_amd import qlora as q

BF = torch.bfloat16


def test_rank_of_half_an_adapter():
    w = q.FP8Weight.empty(96, 128, device="cpu")
    B = torch.zeros(96, 4, dtype=BF)
    with pytest.raises(ValueError, match="A: missing"):
        q._adapter8(w, None, B, BF, B.device)
    assert q._adapter8(w, None, None, BF, B.device) == 0
    for b_gate, b_up in ((B, B), (B, None), (None, B)):
        with pytest.raises(ValueError, match="A_gate and A_up: missing"):
            q._adapters(96, 128, None, b_gate, None, b_up, BF, B.device)
    with pytest.raises(ValueError, match="both adapters or neither"):
        q._adapters(96, 128, B, B, None, None, BF, B.device)
    assert q._adapters(96, 128, None, None, None, None, BF, B.device) == 0


@pytest.mark.gpu
def test_calls_with_half_an_adapter():
    m, n, k, r = 20, 96, 128, 4
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    X, dY, A, B = z(m, k), z(m, n), z(r, k), z(n, r)
    w8, w4 = q.quantize_fp8(torch.ones(n, k, device="cuda")), q.quantize_nf4(torch.ones(n, k, device="cuda"))
    for a, b in ((None, B), (A, None)):
        with pytest.raises(ValueError):
            q.fp8_linear_fwd(w8, X, a, b, 1.0)
        with pytest.raises(ValueError):
            q.fp8_linear_bwd(w8, X, None, dY, a, b, 1.0)
    for lr in ((None, B, None, B), (None, B, None, None), (None, None, None, B), (A, B, None, B), (A, None, A, B),
               (A, B, A, None)):
        with pytest.raises(ValueError):
            q.gated_fwd(w4, w4, X, *lr, 1.0)
        with pytest.raises(ValueError):
            q.gated_bwd(w4, w4, X, None, dY, dY, dY, *lr, 1.0)


def test_workspace_of_another_device():
    cpu, meta = torch.device("cpu"), torch.device("meta")
    ws = torch.empty(256, dtype=torch.uint8)
    assert q._workspace(ws, 0, cpu) is ws and q._workspace(None, 0, cpu) is None
    assert q._workspace(None, 100, cpu).nbytes == 100
    for bad, dev in ((ws, meta), (ws[::2], cpu)):
        with pytest.raises(ValueError, match="ws"):
            q._workspace(bad, 0, dev)


@pytest.mark.gpu
def test_calls_with_a_workspace_in_host_memory():
    m, n, k = 20, 96, 128
    z = lambda *s: torch.zeros(s, dtype=BF, device="cuda")  # noqa: E731
    X, dY, ws = z(m, k), z(m, n), torch.empty(1 << 24, dtype=torch.uint8)
    w8, w4 = q.quantize_fp8(torch.ones(n, k, device="cuda")), q.quantize_nf4(torch.ones(n, k, device="cuda"))
    with pytest.raises(ValueError, match="ws"):
        q.fp8_linear_fwd(w8, X, None, None, 1.0, ws=ws)
    with pytest.raises(ValueError, match="ws"):
        q.fp8_linear_bwd(w8, X, None, dY, None, None, 1.0, ws=ws)
    with pytest.raises(ValueError, match="ws"):
        q.gated_fwd(w4, w4, X, None, None, None, None, 1.0, ws=ws)
    with pytest.raises(ValueError, match="ws"):
        q.gated_bwd(w4, w4, X, None, dY, dY, dY, None, None, None, None, 1.0, ws=ws)
    own = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    assert torch.equal(q.fp8_linear_fwd(w8, X, None, None, 1.0, ws=own)[0], dY)
    assert torch.equal(q.gated_fwd(w4, w4, X, None, None, None, None, 1.0, ws=own)[0], dY)
