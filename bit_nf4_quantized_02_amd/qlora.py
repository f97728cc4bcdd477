"""Thin Python binding over libqlora.so (ctypes).

Argument marshalling only: torch tensors provide device memory and the
current HIP stream; every computation happens in the library's kernels.
Importing this module loads the library and raises ImportError if it has not
been built (``python -m bit_nf4_quantized_02_amd.build``) -- there is no
fallback of any kind.

Names follow the C ABI in include/qlora.h.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m bit_nf4_quantized_02_amd.build`")
_lib = ctypes.CDLL(LIB_PATH)

BLOCK = 64
DQ_BLOCK = 256
MAX_RANK = 128
SCRATCH_BYTES = 64 << 20   # QLORA_SCRATCH_BYTES: the library's own device scratch per device
DT_BF16, DT_FP32, DT_FP16 = 0, 1, 2
FP8_BLOCK = 128    # contraction elements per scale of the 8-bit layer

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_sz = ctypes.c_size_t
_f = ctypes.c_float


class _Weight(ctypes.Structure):
    _fields_ = [("n", _i64), ("k", _i64), ("codes", _vp), ("code8", _vp), ("s2", _vp), ("mean", _vp),
                ("codebook", _vp), ("scale_bf16", ctypes.c_int32)]


class _Weight8(ctypes.Structure):
    _fields_ = [("n", _i64), ("k", _i64), ("codes", _vp), ("scale", _vp)]


class _Rows8(ctypes.Structure):
    _fields_ = [("M", _i64), ("k", _i64), ("codes", _vp), ("scale", _vp)]


class _Param(ctypes.Structure):
    _fields_ = [("theta", _vp), ("theta16", _vp), ("grad", _vp), ("m", _vp), ("v", _vp), ("count", _i64),
                ("grad_dtype", ctypes.c_int32), ("dtype16", ctypes.c_int32)]


class _Table(ctypes.Structure):
    _fields_ = [("chunks", _vp), ("n_chunks", _i64), ("elements", _i64), ("complete", ctypes.c_int32)]


SCALE_FP32, SCALE_DQ, SCALE_BF16 = 0, 1, 2


_W = ctypes.POINTER(_Weight)
_W8 = ctypes.POINTER(_Weight8)
_R8 = ctypes.POINTER(_Rows8)
_P = ctypes.POINTER(_Param)
_T = ctypes.POINTER(_Table)

_SIGS = {
    "qlora_status_string": (ctypes.c_char_p, [_int]),
    "qlora_build_nf4_codebook": (_int, [ctypes.POINTER(_f)]),
    "qlora_nf4_packed_bytes": (_sz, [_i64, _i64]),
    "qlora_nf4_storage_bytes": (_sz, [_i64, _i64, _int]),
    "qlora_build_uniform4_codebook": (_int, [ctypes.POINTER(_f)]),
    "qlora_quantize_workspace_bytes": (_sz, [_i64, _i64]),
    "qlora_quantize_nf4": (_int, [_vp, _int, _W, _vp, _sz, _vp]),
    "qlora_dequant": (_int, [_W, _vp, _vp]),
    "qlora_linear_workspace_bytes": (_sz, [_i64, _i64, _i64, _int, _int]),
    "qlora_linear_fwd": (_int, [_W, _vp, _i64, _vp, _vp, _int, _f, _vp, _vp, _vp, _sz, _vp]),
    "qlora_linear_bwd": (_int, [_W, _vp, _vp, _vp, _i64, _vp, _vp, _int, _f, _vp, _vp, _vp, _int, _vp, _sz, _vp]),
    "qlora_linear_fwd_scratch": (_int, [_W, _vp, _i64, _vp, _vp, _int, _f, _vp, _vp, _vp]),
    "qlora_lora_linear_workspace_bytes": (_sz, [_i64, _i64, _i64, _int, _int]),
    "qlora_lora_linear_fwd": (_int, [_vp, _i64, _i64, _vp, _i64, _vp, _vp, _int, _f, _vp, _vp, _vp, _sz, _vp]),
    "qlora_lora_linear_bwd": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _int, _f, _vp, _vp, _vp, _int,
                                      _vp, _sz, _vp]),
    "qlora_dequant_f16": (_int, [_W, _vp, _vp]),
    "qlora_linear_f16_workspace_bytes": (_sz, [_i64, _i64, _i64, _int, _int]),
    "qlora_linear_fwd_f16": (_int, [_W, _vp, _i64, _vp, _vp, _int, _f, _vp, _vp, _vp, _sz, _vp]),
    "qlora_linear_bwd_f16": (_int, [_W, _vp, _vp, _vp, _i64, _vp, _vp, _int, _f, _vp, _vp, _vp, _int, _vp, _sz,
                                     _vp]),
    "qlora_linear_fwd_dropout": (_int, [_W, _vp, _i64, _vp, _vp, _int, _f, _vp, _f, _vp, _vp, _vp, _sz, _vp]),
    "qlora_linear_bwd_dropout": (_int, [_W, _vp, _vp, _vp, _i64, _vp, _vp, _int, _f, _vp, _f, _vp, _vp, _vp, _int,
                                         _vp, _sz, _vp]),
    "qlora_lowrank_split_cols": (_int, [_int]),
    "qlora_lowrank_project_workspace_bytes": (_sz, [_i64, _i64, _int]),
    "qlora_lowrank_project": (_int, [_vp, _i64, _i64, _vp, _int, _int, _f, _vp, _vp, _vp, _sz, _vp]),
    "qlora_nf4_gemm_fwd": (_int, [_W, _vp, _i64, _vp, _vp, _int, _vp, _vp]),
    "qlora_nf4_gemm_dx": (_int, [_W, _vp, _i64, _vp, _vp, _int, _vp, _vp]),
    "qlora_nf4_gemv_fwd": (_int, [_W, _vp, _i64, _vp, _vp, _int, _f, _vp, _vp, _sz, _vp]),
    "qlora_nf4_gemv_workspace_bytes": (_sz, [_i64]),
    "qlora_nf4_gemv_dx_workspace_bytes": (_sz, [_i64, _i64]),
    "qlora_nf4_gemv_dx": (_int, [_W, _vp, _i64, _vp, _vp, _int, _f, _vp, _vp, _sz, _vp]),
    "qlora_linear_path": (_int, [_i64, _i64, _i64, _int, _int]),
    "qlora_nf4_expand_bytes": (_sz, [_i64, _i64, _int, _int]),
    "qlora_nf4_expand": (_int, [_W, _vp, _int, _int, _vp, _sz, _vp]),
    "qlora_bf16_gemm_workspace_bytes": (_sz, [_i64, _i64, _int, _i64]),
    "qlora_bf16_gemm": (_int, [_vp, _i64, _i64, _vp, _int, _vp, _i64, _vp, _vp, _sz, _vp]),
    "qlora_bf16_gemm_nn": (_int, [_vp, _i64, _i64, _vp, _int, _vp, _i64, _vp, _vp, _sz, _vp]),
    "qlora_lowrank_grad_workspace_bytes": (_sz, [_i64, _i64, _int]),
    "qlora_lowrank_grad": (_int, [_vp, _i64, _i64, _vp, _int, _f, _vp, _int, _int, _vp, _sz, _vp]),
    "qlora_silu_mul_fwd": (_int, [_vp, _vp, _vp, _i64, _vp]),
    "qlora_silu_mul_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _vp]),
    "qlora_adapter_merge": (_int, [_W, _vp, _vp, _int, _f, _vp, _int, _vp]),
    "qlora_adapter_unmerge": (_int, [_vp, _i64, _i64, _vp, _vp, _int, _f, _vp, _vp]),
    "qlora_adamw_step": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _f, _f, _f, _f, _f, _vp]),
    "qlora_gated_workspace_bytes": (_sz, [_i64, _i64, _i64, _int, _int]),
    "qlora_gated_fwd": (_int, [_W, _W, _vp, _i64, _int, _vp, _vp, _vp, _vp, _int, _f, _vp, _vp, _vp, _vp, _vp, _sz,
                               _vp]),
    "qlora_gated_bwd": (_int, [_W, _W, _vp, _vp, _vp, _vp, _vp, _i64, _int, _vp, _vp, _vp, _vp, _int, _f, _vp, _vp, _vp,
                               _vp, _vp, _int, _vp, _sz, _vp]),
    "qlora_fp8_storage_bytes": (_sz, [_i64, _i64]),
    "qlora_quantize_fp8": (_int, [_vp, _int, _W8, _vp]),
    "qlora_dequant_fp8": (_int, [_W8, _vp, _vp]),
    "qlora_fp8_linear_workspace_bytes": (_sz, [_i64, _i64, _i64, _int, _int]),
    "qlora_fp8_linear_fwd": (_int, [_W8, _vp, _i64, _int, _vp, _vp, _int, _f, _vp, _vp, _vp, _sz, _vp]),
    "qlora_fp8_linear_bwd": (_int, [_W8, _vp, _vp, _vp, _i64, _int, _vp, _vp, _int, _f, _vp, _vp, _vp, _int, _vp, _sz,
                                     _vp]),
    "qlora_fp8_rows_bytes": (_sz, [_i64, _i64]),
    "qlora_dequant_fp8_rows": (_int, [_R8, _int, _vp, _vp]),
    "qlora_fp8_linear_rows_workspace_bytes": (_sz, [_i64, _i64, _i64, _int]),
    "qlora_fp8_linear_fwd_rows": (_int, [_W8, _R8, _vp, _int, _vp, _vp, _int, _f, _vp, _vp, _vp, _sz, _vp]),
    "qlora_rms_norm_fwd": (_int, [_vp, _vp, _vp, _int, _i64, _i64, _int, _f, _vp, _vp, _vp, _R8, _vp]),
    "qlora_rms_norm_bwd_workspace_bytes": (_sz, [_i64, _i64]),
    "qlora_rms_norm_bwd": (_int, [_vp, _vp, _vp, _vp, _int, _vp, _i64, _i64, _int, _vp, _vp, _int, _vp, _sz, _vp]),
    "qlora_param_table_bytes": (_sz, [_P, _i64]),
    "qlora_param_table_build": (_int, [_P, _i64, _vp, _sz, _T]),
    "qlora_grad_norm_workspace_bytes": (_sz, []),
    "qlora_grad_norm": (_int, [_T, _f, _f, _vp, _vp, _sz, _vp]),
    "qlora_adamw_step_many": (_int, [_T, _vp, _f, _i64, _f, _f, _f, _f, _f, _vp]),
    "qlora_calib_mfma": (_int, [_int, _int, _vp, _vp]),
    "qlora_calib_stream_read": (_int, [_vp, _i64, _vp, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class QLoraError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} ({status})")
        self.status = status


def status_string(status: int) -> str:
    return _lib.qlora_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != 0:
        raise QLoraError(status, where)


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()  # (every call's argument types are declared)


def _stream(stream=None):
    if stream is None:  # the current stream of the current device (without building its Stream object: 3 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _need(t: torch.Tensor, dtype, shape, name):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on the GPU, "
                         f"got {t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()} device={t.device}")


def _bytes(nbytes: int, device) -> torch.Tensor | None:
    return torch.empty(max(int(nbytes), 0), dtype=torch.uint8, device=device) if nbytes > 0 else None


# --------------------------------------------------------------------------- codebook

def build_nf4_codebook() -> list[float]:
    """The 16 NF4 levels (host, fp32), ascending."""
    buf = (_f * 16)()
    _check(_lib.qlora_build_nf4_codebook(buf), "qlora_build_nf4_codebook")
    return [buf[i] for i in range(16)]


def build_uniform4_codebook() -> list[float]:
    """The 16 levels of the uniform INT4 grid (host, fp32), ascending."""
    buf = (_f * 16)()
    _check(_lib.qlora_build_uniform4_codebook(buf), "qlora_build_uniform4_codebook")
    return [buf[i] for i in range(16)]


def nf4_packed_bytes(n: int, k: int, double_quant: bool = True, scale_dtype=torch.float32) -> int:
    """Bytes of an encoded weight; without double quantization the block
    scales are fp32, or bf16 with scale_dtype=torch.bfloat16."""
    form = SCALE_DQ if double_quant else (SCALE_BF16 if scale_dtype == torch.bfloat16 else SCALE_FP32)
    return int(_lib.qlora_nf4_storage_bytes(n, k, form))


def quantize_workspace_bytes(n: int, k: int) -> int:
    return int(_lib.qlora_quantize_workspace_bytes(n, k))


def linear_workspace_bytes(M: int, n: int, k: int, r: int, is_bwd: bool, dtype=torch.bfloat16) -> int:
    fn = _lib.qlora_linear_f16_workspace_bytes if _is_f16(dtype) else _lib.qlora_linear_workspace_bytes
    return int(fn(M, n, k, r, int(bool(is_bwd))))


def _is_f16(dtype) -> bool:
    """The 16-bit compute type of a layer call: bf16 (default) or fp16."""
    if dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"compute dtype must be torch.bfloat16 or torch.float16, got {dtype}")
    return dtype == torch.float16


# --------------------------------------------------------------------------- weight

@dataclass
class NF4Weight:
    """Device buffers of one encoded [n, k] weight (owned by these tensors)."""
    n: int
    k: int
    codes: torch.Tensor      # uint8 [n, k/2]
    code8: torch.Tensor | None   # uint8 [n*k/64] (None: no double quantization)
    s2: torch.Tensor             # fp32  [ceil(nb/256)], or [nb] fp32 / bf16 block scales without it
    mean: torch.Tensor | None    # fp32  [1]
    codebook: torch.Tensor   # fp32  [16]

    @staticmethod
    def empty(n: int, k: int, device="cuda", codebook: torch.Tensor | None = None,
              double_quant: bool = True, scale_dtype=torch.float32) -> "NF4Weight":
        """Buffers for one encoded weight; without double quantization code8
        and mean are None and s2 holds one scale per block, fp32 or (with
        scale_dtype=torch.bfloat16) bf16."""
        nb = n * k // BLOCK
        nc = -(-nb // DQ_BLOCK)
        if codebook is None:
            codebook = torch.tensor(build_nf4_codebook(), dtype=torch.float32, device=device)
        codes = torch.empty((n, k // 2), dtype=torch.uint8, device=device)
        if not double_quant:
            if scale_dtype not in (torch.float32, torch.bfloat16):
                raise ValueError("block scales are fp32 or bf16")
            return NF4Weight(n, k, codes, None, torch.empty((nb,), dtype=scale_dtype, device=device), None,
                             codebook)
        if scale_dtype != torch.float32:
            raise ValueError("a bf16 block scale is a form without double quantization")
        return NF4Weight(n, k, codes,
                         torch.empty((nb,), dtype=torch.uint8, device=device),
                         torch.empty((nc,), dtype=torch.float32, device=device),
                         torch.empty((1,), dtype=torch.float32, device=device),
                         codebook)

    @property
    def double_quant(self) -> bool:
        return self.code8 is not None

    @property
    def scale_bf16(self) -> bool:
        return self.code8 is None and self.s2.dtype == torch.bfloat16

    def struct(self) -> _Weight:
        p = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        return _Weight(self.n, self.k, self.codes.data_ptr(), p(self.code8), self.s2.data_ptr(),
                       p(self.mean), self.codebook.data_ptr(), int(self.scale_bf16))

    def nbytes(self) -> int:
        return nf4_packed_bytes(self.n, self.k, self.double_quant,
                                torch.bfloat16 if self.scale_bf16 else torch.float32)


def quantize_nf4(W: torch.Tensor, out: NF4Weight | None = None, ws: torch.Tensor | None = None,
                 stream=None, codebook: torch.Tensor | None = None, double_quant: bool = True,
                 scale_dtype=torch.float32) -> NF4Weight:
    """Encode W ([n, k] bf16 or fp32, on the GPU) as 4-bit codes + block
    scales, double-quantized unless double_quant is False (then one fp32, or
    with scale_dtype=torch.bfloat16 one bf16, scale per block); the levels
    are NF4 unless another 16-level device codebook is given (or out's)."""
    if W.dim() != 2:
        raise ValueError("W must be [n, k]")
    n, k = W.shape
    dt = {torch.bfloat16: DT_BF16, torch.float32: DT_FP32}.get(W.dtype)
    if dt is None:
        raise ValueError("W must be bf16 or fp32")
    _need(W, W.dtype, (n, k), "W")
    if out is None:
        out = NF4Weight.empty(n, k, device=W.device, codebook=codebook, double_quant=double_quant,
                              scale_dtype=scale_dtype)
    need = quantize_workspace_bytes(n, k)
    if ws is None:
        ws = _bytes(need, W.device)
    st = out.struct()
    _check(_lib.qlora_quantize_nf4(_ptr(W), dt, ctypes.byref(st), _ptr(ws), 0 if ws is None else ws.numel(),
                                   _stream(stream)), "qlora_quantize_nf4")
    return out


def dequant(w: NF4Weight, out: torch.Tensor | None = None, stream=None, dtype=torch.bfloat16) -> torch.Tensor:
    """[n, k] expansion in bf16 (or fp16), bit-identical to what the GEMM kernels multiply."""
    f16 = _is_f16(dtype)
    if out is None:
        out = torch.empty((w.n, w.k), dtype=dtype, device=w.codes.device)
    _need(out, dtype, (w.n, w.k), "out")
    st = w.struct()
    name = "qlora_dequant_f16" if f16 else "qlora_dequant"
    _check(getattr(_lib, name)(ctypes.byref(st), _ptr(out), _stream(stream)), name)
    return out


# --------------------------------------------------------------------------- linear

def _mask_of(mask: torch.Tensor, M: int, k: int):
    if mask.dtype != torch.uint8 or tuple(mask.shape) != (M, k) or not mask.is_contiguous() or not mask.is_cuda:
        raise ValueError(f"mask: expected contiguous uint8 {(M, k)} on the GPU")
    return _ptr(mask)


def linear_fwd_dropout(w: NF4Weight, X: torch.Tensor, A: torch.Tensor | None, B: torch.Tensor | None, scale: float,
                       mask: torch.Tensor, keep_scale: float, **kw):
    """Y = X W'^T + scale ((X . mask * keep_scale) A^T) B^T (qlora_linear_fwd_dropout);
    the saved T is (X . mask) A^T.  Returns (Y, T)."""
    return linear_fwd(w, X, A, B, scale, _dropout=(mask, keep_scale), **kw)


def linear_bwd_dropout(w: NF4Weight, X: torch.Tensor | None, T: torch.Tensor | None, dY: torch.Tensor,
                       A: torch.Tensor | None, B: torch.Tensor | None, scale: float, mask: torch.Tensor,
                       keep_scale: float, **kw):
    """The gradients of linear_fwd_dropout (qlora_linear_bwd_dropout).  Returns (dX, dA, dB)."""
    return linear_bwd(w, X, T, dY, A, B, scale, _dropout=(mask, keep_scale), **kw)


def linear_fwd(w: NF4Weight, X: torch.Tensor, A: torch.Tensor | None, B: torch.Tensor | None, scale: float,
               Y: torch.Tensor | None = None, T: torch.Tensor | None = None, save_T: bool = True,
               ws: torch.Tensor | None = None, stream=None, _dropout=None, dtype=torch.bfloat16):
    """Y = X W'^T + scale (X A^T) B^T.  Returns (Y, T) with T None unless saved.
    dtype=torch.float16 runs the fp16 layer (qlora_linear_fwd_f16)."""
    M = X.shape[0]
    r = 0 if A is None else A.shape[0]
    f16 = _is_f16(dtype)
    if f16 and _dropout is not None:
        raise ValueError("LoRA dropout runs in bf16 only")
    _need(X, dtype, (M, w.k), "X")
    if r:
        _need(A, dtype, (r, w.k), "A")
        _need(B, dtype, (w.n, r), "B")
    if Y is None:
        Y = torch.empty((M, w.n), dtype=dtype, device=X.device)
    _need(Y, dtype, (M, w.n), "Y")
    if T is None and save_T and r:
        T = torch.empty((M, r), dtype=torch.float32, device=X.device)
    if T is not None:
        _need(T, torch.float32, (M, r), "T")
    st = w.struct()
    if _dropout is not None:
        mp = _mask_of(_dropout[0], M, w.k)
        if ws is None:
            ws = _bytes(linear_workspace_bytes(M, w.n, w.k, r, False), X.device)
        _check(_lib.qlora_linear_fwd_dropout(ctypes.byref(st), _ptr(X), M, _ptr(A), _ptr(B), r, float(scale), mp,
                                             float(_dropout[1]), _ptr(Y), _ptr(T), _ptr(ws),
                                             0 if ws is None else ws.numel(), _stream(stream)),
               "qlora_linear_fwd_dropout")
        return Y, T
    if ws is None:
        ws = _bytes(linear_workspace_bytes(M, w.n, w.k, r, False, dtype), X.device)
    name = "qlora_linear_fwd_f16" if f16 else "qlora_linear_fwd"
    _check(getattr(_lib, name)(ctypes.byref(st), _ptr(X), M, _ptr(A), _ptr(B), r, float(scale), _ptr(Y), _ptr(T),
                               _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)), name)
    return Y, T


def linear_fwd_scratch(w: NF4Weight, X: torch.Tensor, A: torch.Tensor | None, B: torch.Tensor | None,
                       scale: float, Y: torch.Tensor | None = None, T: torch.Tensor | None = None,
                       save_T: bool = True, stream=None):
    """linear_fwd with no workspace (qlora_linear_fwd_scratch): the library's
    own device scratch serves instead, so the call allocates nothing when Y
    (and T, if saved) are given. Calls overlapping on one device race.
    Returns (Y, T)."""
    M = X.shape[0]
    r = 0 if A is None else A.shape[0]
    _need(X, torch.bfloat16, (M, w.k), "X")
    if r:
        _need(A, torch.bfloat16, (r, w.k), "A")
        _need(B, torch.bfloat16, (w.n, r), "B")
    if Y is None:
        Y = torch.empty((M, w.n), dtype=torch.bfloat16, device=X.device)
    _need(Y, torch.bfloat16, (M, w.n), "Y")
    if T is None and save_T and r:
        T = torch.empty((M, r), dtype=torch.float32, device=X.device)
    if T is not None:
        _need(T, torch.float32, (M, r), "T")
    st = w.struct()
    _check(_lib.qlora_linear_fwd_scratch(ctypes.byref(st), _ptr(X), M, _ptr(A), _ptr(B), r, float(scale), _ptr(Y),
                                         _ptr(T), _stream(stream)), "qlora_linear_fwd_scratch")
    return Y, T


def linear_bwd(w: NF4Weight, X: torch.Tensor | None, T: torch.Tensor | None, dY: torch.Tensor,
               A: torch.Tensor | None, B: torch.Tensor | None, scale: float, need_dX: bool = True,
               need_dA: bool = True, need_dB: bool = True, dX: torch.Tensor | None = None,
               dA: torch.Tensor | None = None, dB: torch.Tensor | None = None, accumulate: bool = False,
               ws: torch.Tensor | None = None, stream=None, _dropout=None, dtype=torch.bfloat16):
    """dX = dY W' + s (dY B) A;  dA = s (dY B)^T X;  dB = s dY^T T.  Returns (dX, dA, dB).
    dtype=torch.float16 runs the fp16 layer (qlora_linear_bwd_f16)."""
    M = dY.shape[0]
    r = 0 if A is None else A.shape[0]
    dev = dY.device
    f16 = _is_f16(dtype)
    if f16 and _dropout is not None:
        raise ValueError("LoRA dropout runs in bf16 only")
    _need(dY, dtype, (M, w.n), "dY")
    if X is not None:
        _need(X, dtype, (M, w.k), "X")
    if r:
        _need(A, dtype, (r, w.k), "A")
        _need(B, dtype, (w.n, r), "B")
    if T is not None:
        _need(T, torch.float32, (M, r), "T")
    if need_dX and dX is None:
        dX = torch.empty((M, w.k), dtype=dtype, device=dev)
    if r and need_dA and dA is None:
        dA = (torch.zeros if accumulate else torch.empty)((r, w.k), dtype=torch.float32, device=dev)
    if r and need_dB and dB is None:
        dB = (torch.zeros if accumulate else torch.empty)((w.n, r), dtype=torch.float32, device=dev)
    if dX is not None:
        _need(dX, dtype, (M, w.k), "dX")
    if dA is not None:
        _need(dA, torch.float32, (r, w.k), "dA")
    if dB is not None:
        _need(dB, torch.float32, (w.n, r), "dB")
    st = w.struct()
    if _dropout is not None:
        mp = _mask_of(_dropout[0], M, w.k)
        if ws is None:
            ws = _bytes(linear_workspace_bytes(M, w.n, w.k, r, True), dev)
        _check(_lib.qlora_linear_bwd_dropout(ctypes.byref(st), _ptr(X), _ptr(T), _ptr(dY), M, _ptr(A), _ptr(B), r,
                                             float(scale), mp, float(_dropout[1]), _ptr(dX), _ptr(dA), _ptr(dB),
                                             int(bool(accumulate)), _ptr(ws), 0 if ws is None else ws.numel(),
                                             _stream(stream)), "qlora_linear_bwd_dropout")
        return dX, dA, dB
    if ws is None:
        ws = _bytes(linear_workspace_bytes(M, w.n, w.k, r, True, dtype), dev)
    name = "qlora_linear_bwd_f16" if f16 else "qlora_linear_bwd"
    _check(getattr(_lib, name)(ctypes.byref(st), _ptr(X), _ptr(T), _ptr(dY), M, _ptr(A), _ptr(B), r, float(scale),
                               _ptr(dX), _ptr(dA), _ptr(dB), int(bool(accumulate)), _ptr(ws),
                               0 if ws is None else ws.numel(), _stream(stream)), name)
    return dX, dA, dB


# --------------------------------------------------------------------------- bf16-base LoRA layer

def lora_linear_workspace_bytes(M: int, n: int, k: int, r: int, is_bwd: bool) -> int:
    return int(_lib.qlora_lora_linear_workspace_bytes(M, n, k, r, int(bool(is_bwd))))


def lora_linear_fwd(W: torch.Tensor, X: torch.Tensor, A: torch.Tensor | None, B: torch.Tensor | None, scale: float,
                    Y: torch.Tensor | None = None, T: torch.Tensor | None = None, save_T: bool = True,
                    ws: torch.Tensor | None = None, stream=None):
    """Y = X W^T + scale (X A^T) B^T over a bf16 base W [n, k]
    (qlora_lora_linear_fwd).  Returns (Y, T)."""
    n, k = W.shape
    M = X.shape[0]
    r = 0 if A is None else A.shape[0]
    _need(W, torch.bfloat16, (n, k), "W")
    _need(X, torch.bfloat16, (M, k), "X")
    if r:
        _need(A, torch.bfloat16, (r, k), "A")
        _need(B, torch.bfloat16, (n, r), "B")
    if Y is None:
        Y = torch.empty((M, n), dtype=torch.bfloat16, device=X.device)
    _need(Y, torch.bfloat16, (M, n), "Y")
    if T is None and save_T and r:
        T = torch.empty((M, r), dtype=torch.float32, device=X.device)
    if ws is None:
        ws = _bytes(lora_linear_workspace_bytes(M, n, k, r, False), X.device)
    _check(_lib.qlora_lora_linear_fwd(_ptr(W), n, k, _ptr(X), M, _ptr(A), _ptr(B), r, float(scale), _ptr(Y), _ptr(T),
                                      _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "qlora_lora_linear_fwd")
    return Y, T


def lora_linear_bwd(W: torch.Tensor, X: torch.Tensor | None, T: torch.Tensor | None, dY: torch.Tensor,
                    A: torch.Tensor | None, B: torch.Tensor | None, scale: float, need_dX: bool = True,
                    need_dA: bool = True, need_dB: bool = True, accumulate: bool = False,
                    ws: torch.Tensor | None = None, stream=None):
    """The gradients of lora_linear_fwd (qlora_lora_linear_bwd).  Returns (dX, dA, dB)."""
    n, k = W.shape
    M = dY.shape[0]
    r = 0 if A is None else A.shape[0]
    dev = dY.device
    _need(W, torch.bfloat16, (n, k), "W")
    _need(dY, torch.bfloat16, (M, n), "dY")
    if X is not None:
        _need(X, torch.bfloat16, (M, k), "X")
    if r:
        _need(A, torch.bfloat16, (r, k), "A")
        _need(B, torch.bfloat16, (n, r), "B")
    if T is not None:
        _need(T, torch.float32, (M, r), "T")
    dX = torch.empty((M, k), dtype=torch.bfloat16, device=dev) if need_dX else None
    mk = torch.zeros if accumulate else torch.empty
    dA = mk((r, k), dtype=torch.float32, device=dev) if (r and need_dA) else None
    dB = mk((n, r), dtype=torch.float32, device=dev) if (r and need_dB) else None
    if ws is None:
        ws = _bytes(lora_linear_workspace_bytes(M, n, k, r, True), dev)
    _check(_lib.qlora_lora_linear_bwd(_ptr(W), n, k, _ptr(X), _ptr(T), _ptr(dY), M, _ptr(A), _ptr(B), r, float(scale),
                                      _ptr(dX), _ptr(dA), _ptr(dB), int(bool(accumulate)), _ptr(ws),
                                      0 if ws is None else ws.numel(), _stream(stream)), "qlora_lora_linear_bwd")
    return dX, dA, dB


# --------------------------------------------------------------------------- feed-forward operators

_DT = {torch.bfloat16: DT_BF16, torch.float32: DT_FP32, torch.float16: DT_FP16}


_NOTHING = contextlib.nullcontext()


def _on(stream, device):
    """Context of a call: the tensors' device is current, and what the call
    allocates belongs to the stream that it runs on."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream of {stream.device} for tensors on {device}")
        return torch.cuda.stream(stream)
    if device.index == torch._C._cuda_getDevice():  # (a tensor of the device exists: CUDA is initialised)
        return _NOTHING
    return torch.cuda.device(device)


def _given(t: torch.Tensor | None, dtype, shape, name, device) -> None:
    """_need for an operand that may be left out, on the call's device."""
    if t is None:
        return
    if t.dtype == dtype and t.shape == shape and t.is_cuda and t.device == device and t.is_contiguous():
        return  # (what follows says what is wrong)
    _need(t, dtype, shape, name)
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _out(t: torch.Tensor | None, want: bool, dtype, shape, name, device, zeros: bool = False) -> torch.Tensor | None:
    """An output: the caller's, checked, or a new one where it is wanted."""
    if t is None and want:
        return (torch.zeros if zeros else torch.empty)(shape, dtype=dtype, device=device)
    _given(t, dtype, shape, name, device)
    return t


def _workspace(ws: torch.Tensor | None, nbytes: int, device) -> torch.Tensor | None:
    """The call's workspace: the caller's, on its device and whole (its size is the call's check), or a new one."""
    if ws is None:
        return _bytes(nbytes, device)
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws: expected contiguous on {device}, got contiguous={ws.is_contiguous()} on {ws.device}")
    return ws


# --------------------------------------------------------------------------- gated feed-forward block

def gated_workspace_bytes(M: int, n: int, k: int, r: int, is_bwd: bool) -> int:
    return int(_lib.qlora_gated_workspace_bytes(M, n, k, r, int(bool(is_bwd))))


def _adapters(n, k, A_gate, B_gate, A_up, B_up, dt, dev) -> int:
    """The block's rank; both adapters or neither, of one rank."""
    r = 0 if A_gate is None else A_gate.shape[0]
    if (A_gate is None) != (A_up is None):
        raise ValueError("both adapters or neither")
    if A_gate is None and not (B_gate is None and B_up is None):
        raise ValueError("A_gate and A_up: missing for the B given")
    if r:
        for t, shape, name in ((A_gate, (r, k), "A_gate"), (A_up, (r, k), "A_up"), (B_gate, (n, r), "B_gate"),
                               (B_up, (n, r), "B_up")):
            if t is None:
                raise ValueError(f"{name}: missing")
            _given(t, dt, shape, name, dev)
    return r


def gated_fwd(w_gate: NF4Weight, w_up: NF4Weight, X: torch.Tensor, A_gate: torch.Tensor | None,
              B_gate: torch.Tensor | None, A_up: torch.Tensor | None, B_up: torch.Tensor | None, scale: float,
              H: torch.Tensor | None = None, G: torch.Tensor | None = None, U: torch.Tensor | None = None,
              T: torch.Tensor | None = None, save: bool = True, ws: torch.Tensor | None = None, stream=None):
    """H = silu(G) U with G and U the two layers' outputs, in bf16 or fp16 as X
    (qlora_gated_fwd).  Returns (H, G, U, T): with save, G, U ([M, n]) and T
    ([2, M, r] fp32) for gated_bwd; else those given, or None."""
    M, dt, dev, n, k = X.shape[0], X.dtype, w_gate.codes.device, w_gate.n, w_gate.k
    _is_f16(dt)
    _given(X, dt, (M, k), "X", dev)
    if w_up.codes.device != dev:
        raise ValueError(f"w_up: on {w_up.codes.device}, expected {dev}")
    r = _adapters(n, k, A_gate, B_gate, A_up, B_up, dt, dev)
    sg, su = w_gate.struct(), w_up.struct()
    with _on(stream, dev):
        H = _out(H, True, dt, (M, n), "H", dev)
        G = _out(G, save, dt, (M, n), "G", dev)
        U = _out(U, save, dt, (M, n), "U", dev)
        T = _out(T, save and r > 0, torch.float32, (2, M, r), "T", dev)
        ws = _workspace(ws, gated_workspace_bytes(M, n, k, r, False) if ws is None else 0, dev)
        _check(_lib.qlora_gated_fwd(ctypes.byref(sg), ctypes.byref(su), _ptr(X), M, _DT[dt], _ptr(A_gate), _ptr(B_gate),
                                    _ptr(A_up), _ptr(B_up), r, float(scale), _ptr(H), _ptr(G), _ptr(U), _ptr(T),
                                    _ptr(ws), 0 if ws is None else ws.nbytes, _stream(stream)), "qlora_gated_fwd")
    return H, G, U, T


def gated_bwd(w_gate: NF4Weight, w_up: NF4Weight, X: torch.Tensor | None, T: torch.Tensor | None, G: torch.Tensor,
              U: torch.Tensor, dH: torch.Tensor, A_gate: torch.Tensor | None, B_gate: torch.Tensor | None,
              A_up: torch.Tensor | None, B_up: torch.Tensor | None, scale: float, need_dX: bool = True,
              need_dA: bool = True, need_dB: bool = True, dX: torch.Tensor | None = None,
              dA_gate: torch.Tensor | None = None, dB_gate: torch.Tensor | None = None,
              dA_up: torch.Tensor | None = None, dB_up: torch.Tensor | None = None, accumulate: bool = False,
              ws: torch.Tensor | None = None, stream=None):
    """The gradients of gated_fwd from its saved G, U, T (qlora_gated_bwd).
    Returns (dX, dA_gate, dB_gate, dA_up, dB_up)."""
    M, dt, dev, n, k = dH.shape[0], dH.dtype, w_gate.codes.device, w_gate.n, w_gate.k
    _is_f16(dt)
    for t, shape, name in ((dH, (M, n), "dH"), (G, (M, n), "G"), (U, (M, n), "U"), (X, (M, k), "X")):
        _given(t, dt, shape, name, dev)
    if w_up.codes.device != dev:
        raise ValueError(f"w_up: on {w_up.codes.device}, expected {dev}")
    r = _adapters(n, k, A_gate, B_gate, A_up, B_up, dt, dev)
    if r:
        _given(T, torch.float32, (2, M, r), "T", dev)
    sg, su = w_gate.struct(), w_up.struct()
    f32, a, b = torch.float32, r > 0 and need_dA, r > 0 and need_dB
    with _on(stream, dev):
        dX = _out(dX, need_dX, dt, (M, k), "dX", dev)
        dA_gate = _out(dA_gate, a, f32, (r, k), "dA_gate", dev, zeros=accumulate)
        dB_gate = _out(dB_gate, b, f32, (n, r), "dB_gate", dev, zeros=accumulate)
        dA_up = _out(dA_up, a, f32, (r, k), "dA_up", dev, zeros=accumulate)
        dB_up = _out(dB_up, b, f32, (n, r), "dB_up", dev, zeros=accumulate)
        ws = _workspace(ws, gated_workspace_bytes(M, n, k, r, True) if ws is None else 0, dev)
        _check(_lib.qlora_gated_bwd(ctypes.byref(sg), ctypes.byref(su), _ptr(X), _ptr(T), _ptr(G), _ptr(U), _ptr(dH), M,
                                    _DT[dt], _ptr(A_gate), _ptr(B_gate), _ptr(A_up), _ptr(B_up), r, float(scale),
                                    _ptr(dX), _ptr(dA_gate), _ptr(dB_gate), _ptr(dA_up), _ptr(dB_up),
                                    int(bool(accumulate)), _ptr(ws), 0 if ws is None else ws.nbytes, _stream(stream)),
               "qlora_gated_bwd")
    return dX, dA_gate, dB_gate, dA_up, dB_up


# --------------------------------------------------------------------------- 8-bit layer

@dataclass
class FP8Weight:
    """Device buffers of one 8-bit [n, k] weight (owned by these tensors)."""
    n: int
    k: int
    codes: torch.Tensor      # uint8 E4M3 patterns [n, k up to a multiple of 128]
    scale: torch.Tensor      # uint8 exponent bytes [ceil(n / 128), ceil(k / 128)]

    @staticmethod
    def empty(n: int, k: int, device="cuda") -> "FP8Weight":
        kb = -(-k // FP8_BLOCK)
        return FP8Weight(n, k, torch.empty((n, kb * FP8_BLOCK), dtype=torch.uint8, device=device),
                         torch.empty((-(-n // FP8_BLOCK), kb), dtype=torch.uint8, device=device))

    def struct(self) -> _Weight8:
        kb = -(-self.k // FP8_BLOCK)
        _need(self.codes, torch.uint8, (self.n, kb * FP8_BLOCK), "codes")
        _given(self.scale, torch.uint8, (-(-self.n // FP8_BLOCK), kb), "scale", self.codes.device)
        return self._struct()

    def _struct(self) -> _Weight8:
        return _Weight8(self.n, self.k, self.codes.data_ptr(), self.scale.data_ptr())

    def nbytes(self) -> int:
        return int(_lib.qlora_fp8_storage_bytes(self.n, self.k))


def quantize_fp8(W: torch.Tensor, out: FP8Weight | None = None, stream=None) -> FP8Weight:
    """Encode W ([n, k] bf16, fp16 or fp32, on the GPU) as E4M3 values with one
    power-of-two scale per 128 x 128 tile (qlora_quantize_fp8)."""
    if W.dim() != 2 or W.dtype not in _DT:
        raise ValueError("W must be [n, k] in bf16, fp16 or fp32")
    n, k = W.shape
    _need(W, W.dtype, (n, k), "W")
    with _on(stream, W.device):
        if out is None:
            out = FP8Weight.empty(n, k, device=W.device)
            st = out._struct()
        elif (out.n, out.k) != (n, k):
            raise ValueError(f"out: [{out.n}, {out.k}], expected [{n}, {k}]")
        else:
            st = out.struct()
        _check(_lib.qlora_quantize_fp8(_ptr(W), _DT[W.dtype], ctypes.byref(st), _stream(stream)), "qlora_quantize_fp8")
    return out


def dequant_fp8(w: FP8Weight, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of an 8-bit weight, [n, k] bf16 (qlora_dequant_fp8)."""
    dev = w.codes.device
    st = w.struct()
    with _on(stream, dev):
        out = _out(out, True, torch.bfloat16, (w.n, w.k), "out", dev)
        _check(_lib.qlora_dequant_fp8(ctypes.byref(st), _ptr(out), _stream(stream)), "qlora_dequant_fp8")
    return out


def fp8_linear_workspace_bytes(M: int, n: int, k: int, r: int, is_bwd: bool) -> int:
    return int(_lib.qlora_fp8_linear_workspace_bytes(M, n, k, r, int(bool(is_bwd))))


def _adapter8(w: FP8Weight, A: torch.Tensor | None, B: torch.Tensor | None, dt, dev) -> int:
    """The layer's rank; both factors or neither."""
    r = 0 if A is None else A.shape[0]
    if A is None and B is not None:
        raise ValueError("A: missing for the B given")
    if r:
        if B is None:
            raise ValueError("B: missing")
        _given(A, dt, (r, w.k), "A", dev)
        _given(B, dt, (w.n, r), "B", dev)
    return r


def fp8_linear_fwd(w: FP8Weight, X: torch.Tensor, A: torch.Tensor | None, B: torch.Tensor | None, scale: float,
                   Y: torch.Tensor | None = None, T: torch.Tensor | None = None, save_T: bool = True,
                   ws: torch.Tensor | None = None, stream=None):
    """Y = X8 W8^T + scale (X A^T) B^T with X encoded in the call
    (qlora_fp8_linear_fwd); bf16 or fp16, as X.  Returns (Y, T)."""
    st = w.struct()
    M, dt, dev = X.shape[0], X.dtype, w.codes.device
    _is_f16(dt)
    _given(X, dt, (M, w.k), "X", dev)
    r = _adapter8(w, A, B, dt, dev)
    with _on(stream, dev):
        Y = _out(Y, True, dt, (M, w.n), "Y", dev)
        T = _out(T, save_T and r > 0, torch.float32, (M, r), "T", dev)
        ws = _workspace(ws, fp8_linear_workspace_bytes(M, w.n, w.k, r, False) if ws is None else 0, dev)
        _check(_lib.qlora_fp8_linear_fwd(ctypes.byref(st), _ptr(X), M, _DT[dt], _ptr(A), _ptr(B), r, float(scale),
                                         _ptr(Y), _ptr(T), _ptr(ws), 0 if ws is None else ws.nbytes, _stream(stream)),
               "qlora_fp8_linear_fwd")
    return Y, T


def fp8_linear_bwd(w: FP8Weight, X: torch.Tensor | None, T: torch.Tensor | None, dY: torch.Tensor,
                   A: torch.Tensor | None, B: torch.Tensor | None, scale: float, need_dX: bool = True,
                   need_dA: bool = True, need_dB: bool = True, dX: torch.Tensor | None = None,
                   dA: torch.Tensor | None = None, dB: torch.Tensor | None = None, accumulate: bool = False,
                   ws: torch.Tensor | None = None, stream=None):
    """dX = dY8 W8 + s (dY B) A;  dA = s (dY B)^T X;  dB = s dY^T T
    (qlora_fp8_linear_bwd).  Returns (dX, dA, dB)."""
    st = w.struct()
    M, dt, dev = dY.shape[0], dY.dtype, w.codes.device
    _is_f16(dt)
    _given(dY, dt, (M, w.n), "dY", dev)
    _given(X, dt, (M, w.k), "X", dev)
    r = _adapter8(w, A, B, dt, dev)
    if r:
        _given(T, torch.float32, (M, r), "T", dev)
    with _on(stream, dev):
        dX = _out(dX, need_dX, dt, (M, w.k), "dX", dev)
        dA = _out(dA, r > 0 and need_dA, torch.float32, (r, w.k), "dA", dev, zeros=accumulate)
        dB = _out(dB, r > 0 and need_dB, torch.float32, (w.n, r), "dB", dev, zeros=accumulate)
        ws = _workspace(ws, fp8_linear_workspace_bytes(M, w.n, w.k, r, True) if ws is None else 0, dev)
        _check(_lib.qlora_fp8_linear_bwd(ctypes.byref(st), _ptr(X), _ptr(T), _ptr(dY), M, _DT[dt], _ptr(A), _ptr(B), r,
                                         float(scale), _ptr(dX), _ptr(dA), _ptr(dB), int(bool(accumulate)), _ptr(ws),
                                         0 if ws is None else ws.nbytes, _stream(stream)), "qlora_fp8_linear_bwd")
    return dX, dA, dB


# --------------------------------------------------------------------------- 8-bit activations

@dataclass
class FP8Rows:
    """Device buffers of activations in the 8-bit layer's format (owned by these tensors)."""
    M: int
    k: int
    codes: torch.Tensor      # uint8 E4M3 patterns [M, k up to a multiple of 128]
    scale: torch.Tensor      # uint8 exponent bytes [M, ceil(k / 128)]

    @staticmethod
    def empty(M: int, k: int, device="cuda") -> "FP8Rows":
        kb = -(-k // FP8_BLOCK)
        return FP8Rows(M, k, torch.empty((M, kb * FP8_BLOCK), dtype=torch.uint8, device=device),
                       torch.empty((M, kb), dtype=torch.uint8, device=device))

    def struct(self) -> _Rows8:
        kb = -(-self.k // FP8_BLOCK)
        _need(self.codes, torch.uint8, (self.M, kb * FP8_BLOCK), "codes")
        _given(self.scale, torch.uint8, (self.M, kb), "scale", self.codes.device)
        return self._struct()

    def _struct(self) -> _Rows8:
        return _Rows8(self.M, self.k, self.codes.data_ptr(), self.scale.data_ptr())

    def nbytes(self) -> int:
        return int(_lib.qlora_fp8_rows_bytes(self.M, self.k))


def dequant_fp8_rows(x8: FP8Rows, dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of encoded activations, [M, k] bf16 or fp16 (qlora_dequant_fp8_rows)."""
    _is_f16(dtype)
    st, dev = x8.struct(), x8.codes.device
    with _on(stream, dev):
        out = _out(out, True, dtype, (x8.M, x8.k), "out", dev)
        _check(_lib.qlora_dequant_fp8_rows(ctypes.byref(st), _DT[dtype], _ptr(out), _stream(stream)),
               "qlora_dequant_fp8_rows")
    return out


def fp8_linear_rows_workspace_bytes(M: int, n: int, k: int, r: int) -> int:
    return int(_lib.qlora_fp8_linear_rows_workspace_bytes(M, n, k, r))


def fp8_linear_fwd_rows(w: FP8Weight, x8: FP8Rows, X: torch.Tensor | None, A: torch.Tensor | None,
                        B: torch.Tensor | None, scale: float, Y: torch.Tensor | None = None,
                        T: torch.Tensor | None = None, save_T: bool = True, ws: torch.Tensor | None = None,
                        stream=None, dtype=torch.bfloat16):
    """Y = X8 W8^T + scale (X A^T) B^T on activations that are encoded already
    (qlora_fp8_linear_fwd_rows); X is for the adapter only.  dtype: that of X,
    A, B and Y.  Returns (Y, T)."""
    _is_f16(dtype)
    st, sx = w.struct(), x8.struct()
    M, dev = x8.M, w.codes.device
    if x8.codes.device != dev:
        raise ValueError(f"x8: on {x8.codes.device}, expected {dev}")
    r = _adapter8(w, A, B, dtype, dev)
    if r and X is None:
        raise ValueError("X: missing for the adapter given")
    _given(X, dtype, (M, w.k), "X", dev)
    with _on(stream, dev):
        Y = _out(Y, True, dtype, (M, w.n), "Y", dev)
        T = _out(T, save_T and r > 0, torch.float32, (M, r), "T", dev)
        ws = _workspace(ws, fp8_linear_rows_workspace_bytes(M, w.n, w.k, r) if ws is None else 0, dev)
        _check(_lib.qlora_fp8_linear_fwd_rows(ctypes.byref(st), ctypes.byref(sx), _ptr(X), _DT[dtype], _ptr(A), _ptr(B), r,
                                              float(scale), _ptr(Y), _ptr(T), _ptr(ws), 0 if ws is None else ws.nbytes,
                                              _stream(stream)), "qlora_fp8_linear_fwd_rows")
    return Y, T


# --------------------------------------------------------------------------- residual addition and norm

def _gain(w: torch.Tensor, dt, k: int, dev) -> int:
    """The gain's type: the activations' or fp32."""
    wt = w.dtype
    _given(w, dt if wt != torch.float32 else wt, (k,), "w", dev)
    return _DT[wt]


def rms_norm_fwd(X: torch.Tensor, w: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
                 Y: torch.Tensor | None = None, H: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                 x8: FP8Rows | None = None, want_y: bool = True, want_x8: bool = False, save: bool = True,
                 stream=None):
    """h = X + residual, Y = h rstd w with rstd = (mean(h^2) + eps)^-1/2 over the
    last of X's two dimensions (qlora_rms_norm_fwd); want_x8: Y as the 8-bit
    layer's activations (too).  Returns (Y, h, rstd, x8): h is X itself without a
    residual (H may be `residual`, which is then updated in place), rstd is for
    rms_norm_bwd; Y, rstd and x8 are None unless asked for or given."""
    shape, dt, dev = X.shape, X.dtype, X.device
    if len(shape) != 2:
        raise ValueError("X must be [M, k]")
    M, k = shape
    _is_f16(dt)
    _given(X, dt, shape, "X", dev)
    wt = _gain(w, dt, k, dev)
    if residual is not None:
        _given(residual, dt, shape, "residual", dev)
    elif H is not None:
        raise ValueError("H: given without a residual")
    with _on(stream, dev):
        # (a norm of one token is a kernel of 3 us: empty_like takes half the host's time of empty)
        if Y is not None:
            _given(Y, dt, shape, "Y", dev)
        elif want_y:
            Y = torch.empty_like(X)
        if H is not None:
            _given(H, dt, shape, "H", dev)
        elif residual is not None:
            H = torch.empty_like(X)
        rstd = _out(rstd, save, torch.float32, (M,), "rstd", dev)
        s8 = None
        if x8 is not None:
            if x8.codes.device != dev:
                raise ValueError(f"x8: on {x8.codes.device}, expected {dev}")
            s8 = ctypes.byref(x8.struct())
        elif want_x8:
            x8 = FP8Rows.empty(M, k, device=dev)
            s8 = ctypes.byref(x8._struct())
        _check(_lib.qlora_rms_norm_fwd(X.data_ptr(), _ptr(residual), w.data_ptr(), wt, M, k, _DT[dt], float(eps), _ptr(Y),
                                       _ptr(H), _ptr(rstd), s8, _stream(stream)), "qlora_rms_norm_fwd")
    return Y, X if H is None else H, rstd, x8


def rms_norm_bwd(dY: torch.Tensor, H: torch.Tensor, rstd: torch.Tensor, w: torch.Tensor,
                 dres: torch.Tensor | None = None, need_dX: bool = True, need_dw: bool = True,
                 dX: torch.Tensor | None = None, dw: torch.Tensor | None = None, accumulate: bool = False,
                 ws: torch.Tensor | None = None, stream=None):
    """The gradients of rms_norm_fwd from its h and rstd (qlora_rms_norm_bwd): dX
    of X and the residual alike, with dres, what reaches h past the norm, added
    (dX may be `dres`); dw of the gain, fp32.  Returns (dX, dw)."""
    shape, dt, dev = dY.shape, dY.dtype, dY.device
    if len(shape) != 2:
        raise ValueError("dY must be [M, k]")
    M, k = shape
    _is_f16(dt)
    _given(dY, dt, shape, "dY", dev)
    _given(H, dt, shape, "H", dev)
    _given(rstd, torch.float32, (M,), "rstd", dev)
    _given(dres, dt, shape, "dres", dev)
    wt = _gain(w, dt, k, dev)
    with _on(stream, dev):
        if dX is not None:
            _given(dX, dt, shape, "dX", dev)
        elif need_dX:
            dX = torch.empty_like(dY)
        dw = _out(dw, need_dw, torch.float32, (k,), "dw", dev, zeros=accumulate)
        need = int(_lib.qlora_rms_norm_bwd_workspace_bytes(M, k)) if ws is None and dw is not None else 0
        ws = _workspace(ws, need, dev)
        _check(_lib.qlora_rms_norm_bwd(dY.data_ptr(), H.data_ptr(), rstd.data_ptr(), w.data_ptr(), wt, _ptr(dres), M, k,
                                       _DT[dt], _ptr(dX), _ptr(dw), int(bool(accumulate)), _ptr(ws),
                                       0 if ws is None else ws.nbytes, _stream(stream)), "qlora_rms_norm_bwd")
    return dX, dw


# --------------------------------------------------------------------------- building blocks

def lowrank_split_cols(r: int) -> int:
    return int(_lib.qlora_lowrank_split_cols(r))


def lowrank_project(P: torch.Tensor, Q: torch.Tensor, q_layout: int, scale: float, want_out: bool = True,
                    want_split: bool = False, out: torch.Tensor | None = None, split: torch.Tensor | None = None,
                    ws: torch.Tensor | None = None, stream=None):
    """out = P Q^T (q_layout 0, Q [r, C]) or P Q (q_layout 1, Q [C, r]), fp32; split = bf16 hi/lo of scale*out."""
    M, C = P.shape
    r = Q.shape[0] if q_layout == 0 else Q.shape[1]
    _need(P, torch.bfloat16, (M, C), "P")
    _need(Q, torch.bfloat16, (r, C) if q_layout == 0 else (C, r), "Q")
    if want_out and out is None:
        out = torch.empty((M, r), dtype=torch.float32, device=P.device)
    if want_split and split is None:
        split = torch.empty((M, lowrank_split_cols(r)), dtype=torch.bfloat16, device=P.device)
    if ws is None:
        ws = _bytes(int(_lib.qlora_lowrank_project_workspace_bytes(M, C, r)), P.device)
    _check(_lib.qlora_lowrank_project(_ptr(P), M, C, _ptr(Q), int(q_layout), r, float(scale), _ptr(out), _ptr(split),
                                      _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "qlora_lowrank_project")
    return out, split


def nf4_gemm_fwd(w: NF4Weight, X: torch.Tensor, split: torch.Tensor | None, B: torch.Tensor | None,
                 Y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    M = X.shape[0]
    r = 0 if B is None else B.shape[1]
    if Y is None:
        Y = torch.empty((M, w.n), dtype=torch.bfloat16, device=X.device)
    st = w.struct()
    _check(_lib.qlora_nf4_gemm_fwd(ctypes.byref(st), _ptr(X), M, _ptr(split), _ptr(B), r, _ptr(Y), _stream(stream)),
           "qlora_nf4_gemm_fwd")
    return Y


def nf4_gemm_dx(w: NF4Weight, dY: torch.Tensor, split: torch.Tensor | None, A: torch.Tensor | None,
                dX: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    M = dY.shape[0]
    r = 0 if A is None else A.shape[0]
    if dX is None:
        dX = torch.empty((M, w.k), dtype=torch.bfloat16, device=dY.device)
    st = w.struct()
    _check(_lib.qlora_nf4_gemm_dx(ctypes.byref(st), _ptr(dY), M, _ptr(split), _ptr(A), r, _ptr(dX), _stream(stream)),
           "qlora_nf4_gemm_dx")
    return dX


PATH_GEMV, PATH_FUSED, PATH_EXPANDED = 0, 1, 2


def linear_path(M: int, n: int, k: int, r: int, is_bwd: bool) -> int:
    p = _lib.qlora_linear_path(M, n, k, r, int(is_bwd))
    if p < 0:
        raise QLoraError(-1, "qlora_linear_path")
    return p


def nf4_expand_bytes(n: int, k: int, r: int, transposed: int) -> int:
    return int(_lib.qlora_nf4_expand_bytes(n, k, r, int(transposed)))


def nf4_expand(w: NF4Weight, lr: torch.Tensor | None, r: int, transposed: int, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Expanded bf16 operand: [n, k + xc] (transposed = 0, forward, lr = B),
    [k, np + xc] (1, for dX, lr = A) or [n + xc, k] (2, contraction-major for
    dX, n % 64 == 0, lr = A); returned as a 2-D bf16 tensor."""
    xc = lowrank_split_cols(r)
    transposed = int(transposed)
    if transposed == 1:
        rows, cols = w.k, ((w.n + 63) // 64) * 64 + xc
    elif transposed == 2:
        rows, cols = w.n + xc, w.k
    else:
        rows, cols = w.n, w.k + xc
    nbytes = nf4_expand_bytes(w.n, w.k, r, transposed)
    if out is None:
        out = torch.empty(nbytes // 2, dtype=torch.bfloat16, device=w.codes.device)
    st = w.struct()
    _check(_lib.qlora_nf4_expand(ctypes.byref(st), _ptr(lr), r, int(transposed), _ptr(out), out.numel() * 2,
                                 _stream(stream)), "qlora_nf4_expand")
    return out.view(-1)[: rows * cols].view(rows, cols)


def bf16_gemm_nn(act: torch.Tensor, split: torch.Tensor | None, r: int, F: torch.Tensor, nout: int,
                 out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out = RN_bf16(act F[:kc] + split F[kc:]) over the contraction-major
    operand of nf4_expand(..., transposed=2)."""
    M, kc = act.shape
    if out is None:
        out = torch.empty((M, nout), dtype=torch.bfloat16, device=act.device)
    if ws is None:
        ws = _bytes(bf16_gemm_workspace_bytes(M, kc, r, nout), act.device)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib.qlora_bf16_gemm_nn(_ptr(act), M, kc, _ptr(split), r, _ptr(F), nout, _ptr(out), _ptr(ws), nbytes,
                                   _stream(stream)), "qlora_bf16_gemm_nn")
    return out


def bf16_gemm_workspace_bytes(M: int, kc: int, r: int, nout: int) -> int:
    return int(_lib.qlora_bf16_gemm_workspace_bytes(M, kc, r, nout))


def bf16_gemm(act: torch.Tensor, split: torch.Tensor | None, r: int, F: torch.Tensor, nout: int,
              out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    M, kc = act.shape
    if out is None:
        out = torch.empty((M, nout), dtype=torch.bfloat16, device=act.device)
    if ws is None:
        ws = _bytes(bf16_gemm_workspace_bytes(M, kc, r, nout), act.device)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib.qlora_bf16_gemm(_ptr(act), M, kc, _ptr(split), r, _ptr(F), nout, _ptr(out), _ptr(ws), nbytes,
                                _stream(stream)), "qlora_bf16_gemm")
    return out


def nf4_gemv_workspace_bytes(k: int) -> int:
    return int(_lib.qlora_nf4_gemv_workspace_bytes(k))


def nf4_gemv_fwd(w: NF4Weight, X: torch.Tensor, T: torch.Tensor | None, B: torch.Tensor | None, scale: float,
                 Y: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    M = X.shape[0]
    r = 0 if B is None else B.shape[1]
    if Y is None:
        Y = torch.empty((M, w.n), dtype=torch.bfloat16, device=X.device)
    if ws is None:
        ws = _bytes(nf4_gemv_workspace_bytes(w.k), X.device)
    st = w.struct()
    _check(_lib.qlora_nf4_gemv_fwd(ctypes.byref(st), _ptr(X), M, _ptr(T), _ptr(B), r, float(scale), _ptr(Y),
                                   _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)), "qlora_nf4_gemv_fwd")
    return Y


def nf4_gemv_dx_workspace_bytes(n: int, k: int) -> int:
    return int(_lib.qlora_nf4_gemv_dx_workspace_bytes(n, k))


def nf4_gemv_dx(w: NF4Weight, dY: torch.Tensor, U: torch.Tensor | None, A: torch.Tensor | None, scale: float,
                dX: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dX = dY W' + scale U A for M <= 16 (qlora_nf4_gemv_dx); U = dY B fp32."""
    M = dY.shape[0]
    r = 0 if A is None else A.shape[0]
    if dX is None:
        dX = torch.empty((M, w.k), dtype=torch.bfloat16, device=dY.device)
    if ws is None:
        ws = _bytes(nf4_gemv_dx_workspace_bytes(w.n, w.k), dY.device)
    st = w.struct()
    _check(_lib.qlora_nf4_gemv_dx(ctypes.byref(st), _ptr(dY), M, _ptr(U), _ptr(A), r, float(scale), _ptr(dX),
                                  _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)), "qlora_nf4_gemv_dx")
    return dX


def lowrank_grad(P: torch.Tensor, Q: torch.Tensor, scale: float, g_layout: int, G: torch.Tensor | None = None,
                 accumulate: bool = False, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """G = scale P^T Q as [r, C] (g_layout 0) or [C, r] (g_layout 1), fp32."""
    M, C = P.shape
    r = Q.shape[1]
    if G is None:
        G = (torch.zeros if accumulate else torch.empty)((r, C) if g_layout == 0 else (C, r), dtype=torch.float32,
                                                         device=P.device)
    if ws is None:
        ws = _bytes(int(_lib.qlora_lowrank_grad_workspace_bytes(M, C, r)), P.device)
    _check(_lib.qlora_lowrank_grad(_ptr(P), M, C, _ptr(Q), r, float(scale), _ptr(G), int(g_layout),
                                   int(bool(accumulate)), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "qlora_lowrank_grad")
    return G


class Call:
    """One C-ABI call with its ctypes arguments prebuilt (for tight timing
    loops); calling it only forwards the stored arguments."""

    def __init__(self, name: str, *args, keep=()):
        self.name = name
        self.fn = getattr(_lib, name)
        self.args = args
        self._keep = keep  # keeps ctypes structs referenced by pointer alive

    def __call__(self):
        s = self.fn(*self.args)
        if s != 0:
            raise QLoraError(s, self.name)


# --------------------------------------------------------------------------- MLP join

def silu_mul_fwd(G: torch.Tensor, U: torch.Tensor, H: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _need(U, torch.bfloat16, G.shape, "Up")
    _need(G, torch.bfloat16, G.shape, "G")
    if H is None:
        H = torch.empty_like(G)
    _check(_lib.qlora_silu_mul_fwd(_ptr(G), _ptr(U), _ptr(H), G.numel(), _stream(stream)), "qlora_silu_mul_fwd")
    return H


def silu_mul_bwd(G: torch.Tensor, U: torch.Tensor, dH: torch.Tensor, stream=None):
    for t, nme in ((G, "G"), (U, "Up"), (dH, "dH")):
        _need(t, torch.bfloat16, G.shape, nme)
    dG = torch.empty_like(G)
    dU = torch.empty_like(G)
    _check(_lib.qlora_silu_mul_bwd(_ptr(G), _ptr(U), _ptr(dH), _ptr(dG), _ptr(dU), G.numel(), _stream(stream)),
           "qlora_silu_mul_bwd")
    return dG, dU


def adapter_merge(w: NF4Weight, A: torch.Tensor | None, B: torch.Tensor | None, scale: float,
                  out_dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """round(W' + scale * B A) as a [n, k] bf16 or fp32 tensor."""
    r = 0 if A is None else A.shape[0]
    if r:
        _need(A, torch.bfloat16, (r, w.k), "A")
        _need(B, torch.bfloat16, (w.n, r), "B")
    dt = {torch.bfloat16: 0, torch.float32: 1}[out_dtype]
    if out is None:
        out = torch.empty((w.n, w.k), dtype=out_dtype, device=w.codes.device)
    _need(out, out_dtype, (w.n, w.k), "out")
    st = w.struct()
    _check(_lib.qlora_adapter_merge(ctypes.byref(st), _ptr(A), _ptr(B), r, float(scale), _ptr(out), dt,
                                    _stream(stream)), "qlora_adapter_merge")
    return out


def adapter_unmerge(merged: torch.Tensor, A: torch.Tensor | None, B: torch.Tensor | None, scale: float,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """RN_bf16(merged - scale * B A); out may be `merged` itself."""
    n, k = merged.shape
    r = 0 if A is None else A.shape[0]
    _need(merged, torch.bfloat16, (n, k), "merged")
    if r:
        _need(A, torch.bfloat16, (r, k), "A")
        _need(B, torch.bfloat16, (n, r), "B")
    if out is None:
        out = torch.empty_like(merged)
    _check(_lib.qlora_adapter_unmerge(_ptr(merged), n, k, _ptr(A), _ptr(B), r, float(scale), _ptr(out),
                                      _stream(stream)), "qlora_adapter_unmerge")
    return out


def adamw_step(theta: torch.Tensor, grad: torch.Tensor, m: torch.Tensor, v: torch.Tensor, step: int, lr: float,
               betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.0,
               theta16: torch.Tensor | None = None, stream=None) -> None:
    """In-place AdamW step; m and v may be CPU tensors in pinned memory."""
    n = theta.numel()
    for t, nme in ((theta, "theta"), (grad, "grad")):
        _need(t, torch.float32, theta.shape, nme)
    for t, nme in ((m, "m"), (v, "v")):
        if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous() or not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{nme}: expected contiguous fp32 with {n} elements on the GPU or in pinned host memory")
    if theta16 is not None:
        _need(theta16, torch.bfloat16, theta.shape, "theta16")
    _check(_lib.qlora_adamw_step(_ptr(theta), _ptr(theta16), _ptr(grad), ctypes.c_void_p(m.data_ptr()),
                                 ctypes.c_void_p(v.data_ptr()), n, int(step), float(lr), float(betas[0]),
                                 float(betas[1]), float(eps), float(weight_decay), _stream(stream)),
           "qlora_adamw_step")


@dataclass
class Param:
    """One tensor of a ParamTable: its gradient and, for the step, its fp32
    master copy, moments (on the GPU or in pinned host memory) and 16-bit copy."""
    grad: torch.Tensor
    theta: torch.Tensor | None = None
    m: torch.Tensor | None = None
    v: torch.Tensor | None = None
    theta16: torch.Tensor | None = None

    def _struct(self, dev) -> _Param:
        g, n = self.grad, self.grad.numel()
        if g.dtype not in _DT:
            raise ValueError(f"grad: expected bf16, fp16 or fp32, got {g.dtype}")
        _given(g, g.dtype, g.shape, "grad", dev)
        given = [t is not None for t in (self.theta, self.m, self.v)]
        if any(given) != all(given) or (self.theta16 is not None and not all(given)):
            raise ValueError("theta, m and v: all of them, or only the gradient")
        _given(self.theta, torch.float32, g.shape, "theta", dev)
        for t, name in ((self.m, "m"), (self.v, "v")):
            if t is None:
                continue
            if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous() or not (t.is_cuda or t.is_pinned()):
                raise ValueError(f"{name}: expected contiguous fp32 with {n} elements on the GPU or in pinned host memory")
            if t.is_cuda and t.device != dev:
                raise ValueError(f"{name}: on {t.device}, expected {dev}")
        dt16 = torch.bfloat16
        if self.theta16 is not None:
            dt16 = self.theta16.dtype
            _is_f16(dt16)
            _given(self.theta16, dt16, g.shape, "theta16", dev)
        return _Param(_ptr(self.theta), _ptr(self.theta16), _ptr(g), _ptr(self.m), _ptr(self.v), n, _DT[g.dtype],
                      _DT[dt16])


class ParamTable:
    """The tensors that grad_norm and adamw_step_many work on, laid out once on
    their device (qlora_param_table_build).  It keeps the tensors alive; they are
    the ones that are read and written as long as it is used: a step's gradients
    go into the same buffers as the last one's."""

    def __init__(self, params: list[Param], device=None):
        if device is None:
            device = params[0].grad.device if params else "cuda"
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.params = list(params)
        self.device = device
        arr = (_Param * len(params))(*(p._struct(self.device) for p in params))
        nbytes = int(_lib.qlora_param_table_bytes(arr, len(params)))
        image = torch.empty(nbytes, dtype=torch.uint8)
        self._table = _Table()
        with torch.cuda.device(self.device):
            _check(_lib.qlora_param_table_build(arr, len(params), _ptr(image), nbytes, ctypes.byref(self._table)),
                   "qlora_param_table_build")
            self._chunks = image.to(self.device)
        self._table.chunks = self._chunks.data_ptr() if nbytes else None
        self._ref = ctypes.byref(self._table)

    @property
    def elements(self) -> int:
        return int(self._table.elements)


_GRAD_NORM_WS = int(_lib.qlora_grad_norm_workspace_bytes())


def grad_norm(table: ParamTable, max_norm: float = float("inf"), grad_scale: float = 1.0,
              out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """[norm, factor] on the device, fp32: the norm of grad_scale times all the
    table's gradients, and what scales them to at most max_norm (NaN where a
    gradient is not finite) (qlora_grad_norm)."""
    dev = table.device
    with _on(stream, dev):
        out = _out(out, True, torch.float32, (2,), "out", dev)
        ws = _workspace(ws, _GRAD_NORM_WS, dev)
        _check(_lib.qlora_grad_norm(table._ref, float(grad_scale), float(max_norm), _ptr(out), _ptr(ws), ws.nbytes,
                                    _stream(stream)), "qlora_grad_norm")
    return out


def adamw_step_many(table: ParamTable, step: int, lr: float, betas=(0.9, 0.999), eps: float = 1e-8,
                    weight_decay: float = 0.0, clip: torch.Tensor | None = None, grad_scale: float = 1.0,
                    stream=None) -> None:
    """In-place AdamW step of every tensor in the table, on grad_scale * clip[1]
    times its gradient (qlora_adamw_step_many); clip is grad_norm's result."""
    dev = table.device
    _given(clip, torch.float32, (2,), "clip", dev)
    with _on(stream, dev):
        _check(_lib.qlora_adamw_step_many(table._ref, _ptr(clip), float(grad_scale), int(step), float(lr),
                                          float(betas[0]), float(betas[1]), float(eps), float(weight_decay),
                                          _stream(stream)), "qlora_adamw_step_many")


def calib_mfma(blocks: int, iters: int, sink: torch.Tensor, stream=None) -> int:
    """Enqueue the matrix-core probe; returns its flop count."""
    _need(sink, torch.float32, sink.shape, "sink")
    _check(_lib.qlora_calib_mfma(blocks, iters, _ptr(sink), _stream(stream)), "qlora_calib_mfma")
    return blocks * 8 * iters * 8 * 32768


def calib_stream_read(buf: torch.Tensor, sink: torch.Tensor, stream=None) -> int:
    """Enqueue one streaming read of `buf`; returns the bytes read."""
    nbytes = buf.numel() * buf.element_size()
    _check(_lib.qlora_calib_stream_read(_ptr(buf), nbytes, _ptr(sink), _stream(stream)), "qlora_calib_stream_read")
    return nbytes


def raw():
    """The ctypes handle, for tests that call the C ABI directly."""
    return _lib
