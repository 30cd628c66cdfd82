"""ctypes binding of libqlora (the C ABI in include/qlora.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch provides device memory and the current stream; outputs and
workspaces that the caller does not pass are allocated here with torch, for the
stream the call launches on (the library itself never allocates).  There is no CPU fallback: if the shared
library is missing or a call fails, a ``QLoRAError`` is raised.
"""
import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqlora.so")

QLORA_OK = 0
QLORA_ERR_NULL = -1
QLORA_ERR_SHAPE = -2
QLORA_ERR_ALIGN = -3
QLORA_ERR_WORKSPACE = -4
QLORA_ERR_CUDA = -5
QLORA_ERR_DEVICE = -6
QLORA_ERR_CODEBOOK = -7
QLORA_ERR_FORMAT = -8

# 4-bit codebooks (the weight's `codebook`): NF4 and the FP4 / INT4 baselines.
QLORA_CODEBOOK_NF4 = 0
QLORA_CODEBOOK_FP4 = 1
QLORA_CODEBOOK_INT4 = 2
CODEBOOKS = {"nf4": QLORA_CODEBOOK_NF4, "fp4": QLORA_CODEBOOK_FP4, "int4": QLORA_CODEBOOK_INT4}

# Storage formats of the double-quantized absmax (the weight's `dq_format`):
# unsigned linear 8-bit codes, or E4M3 offsets from the tensor mean.
QLORA_DQ_LINEAR8 = 0
QLORA_DQ_FP8_MEAN = 1
DQ_FORMATS = {"linear8": QLORA_DQ_LINEAR8, "fp8_mean": QLORA_DQ_FP8_MEAN}

# Bits of the device error word (qlora_poll_device_error).
QLORA_DEVERR_OPERANDS = 1 << 0
QLORA_DEVERR_WEIGHT_TILE = 1 << 1
QLORA_DEVERR_FREE_STAGE = 1 << 2
QLORA_DEVERR_ACCUMULATOR = 1 << 3
QLORA_DEVERR_DRAIN = 1 << 4
QLORA_DEVERR_SELFTEST = 1 << 5

QLORA_OP_FWD = 0
QLORA_OP_BWD_DX = 1
QLORA_OP_LORA_BWD = 2

BLOCK = 64
GROUP = 256


class QLoRAError(RuntimeError):
    def __init__(self, fn: str, status: int, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        msg = lib().qlora_status_string(status).decode()
        if status == QLORA_ERR_CUDA:
            msg += f" (cudaError {cuda_error})"
        super().__init__(f"{fn}: {msg}")


class NF4WeightC(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("absmax_q", ctypes.c_void_p),
                ("group_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("block", ctypes.c_int32), ("group", ctypes.c_int32), ("codebook", ctypes.c_int32),
                ("dq_format", ctypes.c_int32)]


class Act8C(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("m", ctypes.c_int64), ("k", ctypes.c_int64)]


class AdapterSetC(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("count", ctypes.c_int32),
                ("r", ctypes.c_int32)]


_LIB = None

_SIGNATURES = {
    "qlora_quantize_nf4_dq": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_quantize_4bit_dq": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p]),
    "qlora_quantize_4bit_dq_format": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                     ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                     ctypes.c_void_p]),
    "qlora_codebook_levels": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(ctypes.c_float)]),
    "qlora_dequant": (ctypes.c_int, [ctypes.POINTER(NF4WeightC), ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_merge_adapter": (ctypes.c_int, [ctypes.POINTER(NF4WeightC), ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_int32, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p]),
    "qlora_linear_fwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(NF4WeightC),
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_float,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_linear_bwd_dx": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(NF4WeightC),
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_float,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_lora_bwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                      ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                ctypes.c_int32]),
    "qlora_last_cuda_error": (ctypes.c_int, []),
    "qlora_poll_device_error": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint)]),
    "qlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "qlora_nf4_levels": (None, [ctypes.POINTER(ctypes.c_float)]),
    "qlora_version": (ctypes.c_int, []),
    "qlora_set_profile_events": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_launch_count": (ctypes.c_uint64, []),
    "qlora_linear_fwd_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(NF4WeightC),
                                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_float,
                                                ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_linear_bwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.POINTER(NF4WeightC), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                        ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_lora_dropout": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_float,
                                          ctypes.c_uint64, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_linear_fwd_dropout": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(NF4WeightC),
                                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_float,
                                                ctypes.c_float, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_void_p,
                                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_linear_bwd_dx_dropout": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(NF4WeightC),
                                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_float,
                                                   ctypes.c_float, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_void_p,
                                                   ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_act_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_act_dequant": (ctypes.c_int, [ctypes.POINTER(Act8C), ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_linear_bwd_act8": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(Act8C), ctypes.c_void_p, ctypes.c_int64,
                                             ctypes.POINTER(NF4WeightC), ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_int32, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_linear_fwd_multi": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(NF4WeightC),
                                              ctypes.POINTER(AdapterSetC), ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_linear_bwd_multi": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Act8C), ctypes.c_void_p,
                                              ctypes.c_int64, ctypes.POINTER(NF4WeightC), ctypes.POINTER(AdapterSetC),
                                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_multi_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                      ctypes.c_int32, ctypes.c_int32]),
    "qlora_selftest_bounded_wait": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_selftest_div255": (ctypes.c_int, [ctypes.c_uint32, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_void_p]),
}


def lib() -> ctypes.CDLL:
    """Load libqlora.so from the package directory (built in-tree)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m bit_nf4_quantized_qlora_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def _check(fn: str, status: int) -> None:
    if status != QLORA_OK:
        raise QLoRAError(fn, status, lib().qlora_last_cuda_error() if status == QLORA_ERR_CUDA else 0)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _empty(shape, dtype: torch.dtype, device, stream=None) -> torch.Tensor:
    """What a call allocates, from the pool of the stream it launches on.  A
    block of the current stream's pool would go back to it as soon as the call
    drops the tensor, and could still be in use there when the call starts."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)        # 0 and 1 name the default stream
        stream = (torch.cuda.default_stream(device) if handle in (0, 1)
                  else torch.cuda.ExternalStream(handle, device=device))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _need_cuda(*ts: Optional[torch.Tensor]) -> None:
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


@dataclass
class NF4Weight:
    """A quantized weight: packed codes, absmax codes and group scales (all on
    the device) plus its shape [n x k]."""
    codes: torch.Tensor          # uint8 [n*k/2]
    absmax_q: torch.Tensor       # uint8 [n*k/64]
    group_scale: torch.Tensor    # float32 [ceil(n*k/64/256)] (+ the mean, QLORA_DQ_FP8_MEAN)
    n: int
    k: int
    codebook: int = QLORA_CODEBOOK_NF4
    dq_format: int = QLORA_DQ_LINEAR8

    def c_struct(self) -> NF4WeightC:
        return NF4WeightC(self.codes.data_ptr(), self.absmax_q.data_ptr(), self.group_scale.data_ptr(),
                          self.n, self.k, BLOCK, GROUP, self.codebook, self.dq_format)

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.absmax_q.numel() + 4 * self.group_scale.numel()


def n_groups(numel: int) -> int:
    return (numel // BLOCK + GROUP - 1) // GROUP


def qlora_workspace_bytes(op: int, m: int, n: int, k: int, r: int) -> int:
    return int(lib().qlora_workspace_bytes(op, m, n, k, r))


def qlora_nf4_levels() -> list:
    buf = (ctypes.c_float * 16)()
    lib().qlora_nf4_levels(buf)
    return [float(v) for v in buf]


def qlora_codebook_levels(codebook: int) -> list:
    buf = (ctypes.c_float * 16)()
    _check("qlora_codebook_levels", lib().qlora_codebook_levels(codebook, buf))
    return [float(v) for v in buf]


def qlora_set_profile_events(start: Optional[torch.cuda.Event], stop: Optional[torch.cuda.Event]) -> None:
    """Record `start`/`stop` around the main kernel of the following linear
    calls on this thread (None, None clears)."""
    a = None if start is None else start.cuda_event
    b = None if stop is None else stop.cuda_event
    _check("qlora_set_profile_events", lib().qlora_set_profile_events(a, b))


def qlora_launch_count() -> int:
    return int(lib().qlora_launch_count())


def qlora_poll_device_error(stream=None) -> int:
    flags = ctypes.c_uint(0)
    _check("qlora_poll_device_error", lib().qlora_poll_device_error(_stream(stream), ctypes.byref(flags)))
    return int(flags.value)


def qlora_quantize_nf4_dq(W: torch.Tensor, absmax_fp32: Optional[torch.Tensor] = None,
                          out: Optional[NF4Weight] = None, stream=None) -> NF4Weight:
    """fp32 W [n x k] on the device -> NF4Weight."""
    return qlora_quantize_4bit_dq(W, QLORA_CODEBOOK_NF4, absmax_fp32, out, stream)


def qlora_quantize_4bit_dq(W: torch.Tensor, codebook: int, absmax_fp32: Optional[torch.Tensor] = None,
                           out: Optional[NF4Weight] = None, stream=None,
                           dq_format: int = QLORA_DQ_LINEAR8) -> NF4Weight:
    """fp32 W [n x k] on the device -> NF4Weight in `codebook` (QLORA_CODEBOOK_*)
    with its absmax stored in `dq_format` (QLORA_DQ_*)."""
    _need_cuda(W, absmax_fp32)
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a 2-D float32 tensor")
    n, k = W.shape
    numel = n * k
    n_scales = max(n_groups(numel), 1) + (1 if dq_format == QLORA_DQ_FP8_MEAN else 0)
    if out is None:
        dev = W.device
        out = NF4Weight(_empty(numel // 2, torch.uint8, dev, stream), _empty(numel // BLOCK, torch.uint8, dev, stream),
                        _empty(n_scales, torch.float32, dev, stream), n, k, codebook, dq_format)
    else:
        if out.group_scale.numel() < n_scales:
            raise ValueError(f"out.group_scale holds {out.group_scale.numel()} entries, {n_scales} needed")
        out.codebook = codebook
        out.dq_format = dq_format
    _check("qlora_quantize_4bit_dq_format",
           lib().qlora_quantize_4bit_dq_format(W.data_ptr(), n, k, codebook, dq_format, out.codes.data_ptr(),
                                               out.absmax_q.data_ptr(), out.group_scale.data_ptr(),
                                               _ptr(absmax_fp32), _stream(stream)))
    return out


def qlora_dequant(w: NF4Weight, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """NF4Weight -> bf16 W^ [n x k]."""
    if out is None:
        out = _empty((w.n, w.k), torch.bfloat16, w.codes.device, stream)
    _need_cuda(out)
    ws = w.c_struct()
    _check("qlora_dequant", lib().qlora_dequant(ctypes.byref(ws), out.data_ptr(), _stream(stream)))
    return out


def qlora_merge_adapter(w: NF4Weight, A: Optional[torch.Tensor], B: Optional[torch.Tensor], r: int,
                        scale: float, out_bf16: Optional[torch.Tensor] = None, out_f32: Optional[torch.Tensor] = None,
                        want_bf16: bool = True, want_f32: bool = False, stream=None):
    """W' = W^ + scale . B . A [n x k]; returns (bf16 or None, fp32 or None)."""
    A, B, r = _lora_args(A, B, r)
    dev = w.codes.device
    if out_bf16 is None and want_bf16:
        out_bf16 = _empty((w.n, w.k), torch.bfloat16, dev, stream)
    if out_f32 is None and want_f32:
        out_f32 = _empty((w.n, w.k), torch.float32, dev, stream)
    _need_cuda(A, B, out_bf16, out_f32)
    ws = w.c_struct()
    _check("qlora_merge_adapter",
           lib().qlora_merge_adapter(ctypes.byref(ws), _ptr(A), _ptr(B), r, float(scale), _ptr(out_bf16),
                                     _ptr(out_f32), _stream(stream)))
    return out_bf16, out_f32


def _lora_args(A, B, r):
    if A is None or B is None or r == 0:
        return None, None, 0
    return A, B, r


def _workspace(op, m, n, k, r, ws, device, stream):
    need = qlora_workspace_bytes(op, m, n, k, r)
    if ws is None and need > 0:
        ws = _empty(need, torch.uint8, device, stream)
    return ws, (ws.numel() * ws.element_size() if ws is not None else 0)


def qlora_linear_fwd(X: torch.Tensor, w: NF4Weight, A: Optional[torch.Tensor] = None,
                     B: Optional[torch.Tensor] = None, r: int = 0, scale: float = 0.0,
                     out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """Y = bf16(X . W^T + bf16(s X A^T) . B^T); X bf16 [m x k]."""
    A, B, r = _lora_args(A, B, r)
    _need_cuda(X, A, B, out, ws)
    m = X.shape[0]
    if out is None:
        out = _empty((m, w.n), torch.bfloat16, X.device, stream)
    ws, ws_bytes = _workspace(QLORA_OP_FWD, m, w.n, w.k, r, ws, X.device, stream)
    ws_c = w.c_struct()
    _check("qlora_linear_fwd",
           lib().qlora_linear_fwd(X.data_ptr(), m, ctypes.byref(ws_c), _ptr(A), _ptr(B), r, float(scale),
                                  out.data_ptr(), _ptr(ws), ws_bytes, _stream(stream)))
    return out


def qlora_linear_bwd_dx(dY: torch.Tensor, w: NF4Weight, A: Optional[torch.Tensor] = None,
                        B: Optional[torch.Tensor] = None, r: int = 0, scale: float = 0.0,
                        out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """dX = bf16(dY . W^ + bf16(s dY B) . A); dY bf16 [m x n]."""
    A, B, r = _lora_args(A, B, r)
    _need_cuda(dY, A, B, out, ws)
    m = dY.shape[0]
    if out is None:
        out = _empty((m, w.k), torch.bfloat16, dY.device, stream)
    ws, ws_bytes = _workspace(QLORA_OP_BWD_DX, m, w.n, w.k, r, ws, dY.device, stream)
    ws_c = w.c_struct()
    _check("qlora_linear_bwd_dx",
           lib().qlora_linear_bwd_dx(dY.data_ptr(), m, ctypes.byref(ws_c), _ptr(A), _ptr(B), r, float(scale),
                                     out.data_ptr(), _ptr(ws), ws_bytes, _stream(stream)))
    return out


def qlora_lora_bwd(X: torch.Tensor, dY: torch.Tensor, A: torch.Tensor, B: torch.Tensor, r: int, scale: float,
                   dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dA, dB) = (bf16(U^T X), bf16(dY^T T)) with U = bf16(s dY B), T = bf16(s X A^T)."""
    _need_cuda(X, dY, A, B, dA, dB, ws)
    m, k = X.shape
    n = dY.shape[1]
    if dA is None:
        dA = _empty((r, k), torch.bfloat16, X.device, stream)
    if dB is None:
        dB = _empty((n, r), torch.bfloat16, X.device, stream)
    ws, ws_bytes = _workspace(QLORA_OP_LORA_BWD, m, n, k, r, ws, X.device, stream)
    _check("qlora_lora_bwd",
           lib().qlora_lora_bwd(X.data_ptr(), dY.data_ptr(), m, n, k, A.data_ptr(), B.data_ptr(), r, float(scale),
                                dA.data_ptr(), dB.data_ptr(), _ptr(ws), ws_bytes, _stream(stream)))
    return dA, dB


def qlora_linear_bwd(dY: torch.Tensor, X: torch.Tensor, w: NF4Weight, A: torch.Tensor, B: torch.Tensor, r: int,
                     scale: float, T: Optional[torch.Tensor] = None, dX: Optional[torch.Tensor] = None,
                     dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None, want_dx: bool = True,
                     ws: Optional[torch.Tensor] = None, stream=None):
    """(dX or None, dA, dB) of the layer in one call; T = the forward's
    bf16(s X A^T) (the first m*r*2 bytes of its workspace, which may be `ws`)
    or None."""
    _need_cuda(dY, X, A, B, T, dX, dA, dB, ws)
    m, k = X.shape
    n = dY.shape[1]
    if dX is None and want_dx:
        dX = _empty((m, k), torch.bfloat16, X.device, stream)
    if dA is None:
        dA = _empty((r, k), torch.bfloat16, X.device, stream)
    if dB is None:
        dB = _empty((n, r), torch.bfloat16, X.device, stream)
    ws, ws_bytes = _workspace(QLORA_OP_LORA_BWD, m, n, k, r, ws, X.device, stream)
    ws_c = w.c_struct()
    _check("qlora_linear_bwd",
           lib().qlora_linear_bwd(dY.data_ptr(), X.data_ptr(), _ptr(T), m, ctypes.byref(ws_c), A.data_ptr(),
                                  B.data_ptr(), r, float(scale), _ptr(dX), dA.data_ptr(), dB.data_ptr(), _ptr(ws),
                                  ws_bytes, _stream(stream)))
    return dX, dA, dB


def qlora_lora_dropout(X: torch.Tensor, p: float, seed: int, offset: int, out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """Xd = bf16(D . X . fp32(1 / fp32(1 - p))) with the counter-based keep
    mask of (seed, offset); X bf16 [m x k]."""
    _need_cuda(X, out)
    m, k = X.shape
    if out is None:
        out = _empty(X.shape, X.dtype, X.device, stream)
    _check("qlora_lora_dropout", lib().qlora_lora_dropout(X.data_ptr(), m, k, float(p), int(seed), int(offset),
                                                          out.data_ptr(), _stream(stream)))
    return out


def qlora_linear_fwd_dropout(X: torch.Tensor, w: NF4Weight, A: torch.Tensor, B: torch.Tensor, r: int, scale: float,
                             p: float, seed: int, offset: int, out: Optional[torch.Tensor] = None,
                             Xd: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(Y, Xd): Y = bf16(X . W^T + bf16(s Xd A^T) . B^T) with Xd the dropout of X."""
    _need_cuda(X, A, B, out, Xd, ws)
    m = X.shape[0]
    if out is None:
        out = _empty((m, w.n), torch.bfloat16, X.device, stream)
    if Xd is None:
        Xd = _empty(X.shape, X.dtype, X.device, stream)
    ws, ws_bytes = _workspace(QLORA_OP_FWD, m, w.n, w.k, r, ws, X.device, stream)
    ws_c = w.c_struct()
    _check("qlora_linear_fwd_dropout",
           lib().qlora_linear_fwd_dropout(X.data_ptr(), m, ctypes.byref(ws_c), _ptr(A), _ptr(B), r, float(scale),
                                          float(p), int(seed), int(offset), Xd.data_ptr(), out.data_ptr(), _ptr(ws),
                                          ws_bytes, _stream(stream)))
    return out, Xd


def qlora_linear_bwd_dx_dropout(dY: torch.Tensor, w: NF4Weight, A: torch.Tensor, B: torch.Tensor, r: int,
                                scale: float, p: float, seed: int, offset: int, out: Optional[torch.Tensor] = None,
                                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dX = bf16(bf16(dY . W^) + D . (U . A) . fp32(1 / fp32(1 - p))), U = bf16(s dY B)."""
    _need_cuda(dY, A, B, out, ws)
    m = dY.shape[0]
    if out is None:
        out = _empty((m, w.k), torch.bfloat16, dY.device, stream)
    ws, ws_bytes = _workspace(QLORA_OP_BWD_DX, m, w.n, w.k, r, ws, dY.device, stream)
    ws_c = w.c_struct()
    _check("qlora_linear_bwd_dx_dropout",
           lib().qlora_linear_bwd_dx_dropout(dY.data_ptr(), m, ctypes.byref(ws_c), _ptr(A), _ptr(B), r, float(scale),
                                             float(p), int(seed), int(offset), out.data_ptr(), _ptr(ws), ws_bytes,
                                             _stream(stream)))
    return out


def qlora_linear_fwd_noalloc(X: torch.Tensor, w: NF4Weight, A: Optional[torch.Tensor] = None,
                             B: Optional[torch.Tensor] = None, r: int = 0, scale: float = 0.0,
                             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Forward without a workspace: the library's built-in device scratch
    (QLORA_NOALLOC_SCRATCH_BYTES) holds T.  For callers that cannot allocate;
    `out` must then be passed in."""
    A, B, r = _lora_args(A, B, r)
    _need_cuda(X, A, B, out)
    m = X.shape[0]
    if out is None:
        out = _empty((m, w.n), torch.bfloat16, X.device, stream)
    ws_c = w.c_struct()
    _check("qlora_linear_fwd_noalloc",
           lib().qlora_linear_fwd_noalloc(X.data_ptr(), m, ctypes.byref(ws_c), _ptr(A), _ptr(B), r, float(scale),
                                          out.data_ptr(), _stream(stream)))
    return out


@dataclass
class Act8:
    """An 8-bit activation checkpoint of a bf16 tensor [m x k]."""
    codes: torch.Tensor          # int8 [m, k]
    scale: torch.Tensor          # bfloat16 [m, k/64]
    m: int
    k: int

    @classmethod
    def empty(cls, m: int, k: int, device, stream=None) -> "Act8":
        return cls(_empty((m, k), torch.int8, device, stream), _empty((m, k // BLOCK), torch.bfloat16, device, stream),
                   m, k)

    def c_struct(self) -> Act8C:
        return Act8C(self.codes.data_ptr(), self.scale.data_ptr(), self.m, self.k)

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + 2 * self.scale.numel()


def _need(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape, device: torch.device) -> None:
    """The tensor is a contiguous tensor of this type and shape on this device
    (which _stream_on then finds to be the current CUDA device)."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        return
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {list(shape)}, not {t.dtype} {list(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, not on {device}")


def _need_act8(act: Act8, m: int, k: int, device) -> None:
    if act.m != m or act.k != k:
        raise ValueError(f"the checkpoint holds [{act.m} x {act.k}], not [{m} x {k}]")
    codes, scale = act.codes, act.scale
    if not (codes.dtype is torch.int8 and scale.dtype is torch.bfloat16 and codes.shape == (m, k)
            and scale.shape == (m, k // BLOCK) and codes.device == device and scale.device == device
            and codes.is_contiguous() and scale.is_contiguous()):
        _need(codes, "codes", torch.int8, (m, k), device)
        _need(scale, "scale", torch.bfloat16, (m, k // BLOCK), device)


def _need_weight(w: NF4Weight, device) -> None:
    if w.codes.device != device:
        raise ValueError(f"the weight is on {w.codes.device}, not on {device}")


def _out(t: Optional[torch.Tensor], shape, device, stream) -> torch.Tensor:
    return _empty(shape, torch.bfloat16, device, stream) if t is None else t


def _need_ws(ws: Optional[torch.Tensor], device) -> None:
    if ws is not None and (ws.device != device or not ws.is_contiguous()):
        _need_cuda(ws)
        raise ValueError(f"ws is on {ws.device}, not on {device}")


def _stream_on(device: torch.device, stream) -> Optional[int]:
    """The stream's handle; the default is the current stream of the tensors'
    device, which must be the current device (the library launches there)."""
    if device.type != "cuda":
        raise ValueError("tensors must be contiguous CUDA tensors")
    if device.index != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else _stream(stream)


def qlora_act_quantize(X: torch.Tensor, out: Optional[Act8] = None, stream=None) -> Act8:
    """X bf16 [m x k] -> its 8-bit checkpoint: per 64 elements of a row
    scale = bf16(max|x| / 127), codes = rint(x / scale)."""
    if X.dim() != 2 or X.shape[1] % BLOCK:
        raise ValueError("X must be a 2-D tensor with a row length that is a multiple of 64")
    (m, k), dev = X.shape, X.device
    if X.dtype is not torch.bfloat16 or not X.is_contiguous():
        _need(X, "X", torch.bfloat16, (m, k), dev)
    if out is None:
        out = Act8.empty(m, k, dev, stream)
    _need_act8(out, m, k, dev)
    _check("qlora_act_quantize", lib().qlora_act_quantize(X.data_ptr(), m, k, out.codes.data_ptr(),
                                                          out.scale.data_ptr(), _stream_on(dev, stream)))
    return out


def qlora_act_dequant(act: Act8, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The checkpoint's X^ = bf16(codes . scale) [m x k]."""
    dev = act.codes.device
    _need_act8(act, act.m, act.k, dev)
    out = _out(out, (act.m, act.k), dev, stream)
    _need(out, "out", torch.bfloat16, (act.m, act.k), dev)
    a = act.c_struct()
    _check("qlora_act_dequant", lib().qlora_act_dequant(ctypes.byref(a), out.data_ptr(), _stream_on(dev, stream)))
    return out


def qlora_linear_bwd_act8(dY: torch.Tensor, act: Act8, w: NF4Weight, A: torch.Tensor, B: torch.Tensor, r: int,
                          scale: float, T: torch.Tensor, dX: Optional[torch.Tensor] = None,
                          dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None, want_dx: bool = True,
                          ws: Optional[torch.Tensor] = None, stream=None):
    """(dX or None, dA, dB) as qlora_linear_bwd with X read from its 8-bit
    checkpoint; T = the forward's bf16(s X A^T) [m x r]."""
    m, n, k, dev, bf = dY.shape[0], w.n, w.k, dY.device, torch.bfloat16
    if dX is not None or want_dx:
        dX = _out(dX, (m, k), dev, stream)
    dA, dB = _out(dA, (r, k), dev, stream), _out(dB, (n, r), dev, stream)
    for t, name, shape in ((dY, "dY", (m, n)), (A, "A", (r, k)), (B, "B", (n, r)), (T, "T", (m, r)),
                           (dX, "dX", (m, k)), (dA, "dA", (r, k)), (dB, "dB", (n, r))):
        _need(t, name, bf, shape, dev)
    _need_act8(act, m, k, dev)
    _need_weight(w, dev)
    ws, ws_bytes = _workspace(QLORA_OP_LORA_BWD, m, n, k, r, ws, dev, stream)
    _need_ws(ws, dev)
    w_c, a_c = w.c_struct(), act.c_struct()
    _check("qlora_linear_bwd_act8",
           lib().qlora_linear_bwd_act8(dY.data_ptr(), ctypes.byref(a_c), _ptr(T), m, ctypes.byref(w_c), A.data_ptr(),
                                       B.data_ptr(), r, float(scale), _ptr(dX), dA.data_ptr(), dB.data_ptr(), _ptr(ws),
                                       ws_bytes, _stream_on(dev, stream)))
    return dX, dA, dB


def qlora_multi_workspace_bytes(op: int, m: int, n: int, k: int, r: int, count: int) -> int:
    return int(lib().qlora_multi_workspace_bytes(op, m, n, k, r, count))


def _adapter_set(A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor, ids: torch.Tensor, m: int, w: NF4Weight, dev):
    if A.dim() != 3:
        raise ValueError("A must be a 3-D tensor [count x r x k]")
    count, r, k = A.shape
    bf = torch.bfloat16
    # One condition for the call that is right; the checks that name what is
    # wrong cost a call each.
    if not (A.dtype is bf and B.dtype is bf and scale.dtype is torch.float32 and ids.dtype is torch.int32
            and k == w.k and B.shape == (count, w.n, r) and scale.shape == (count,) and ids.shape == (m,)
            and A.device == dev and B.device == dev and scale.device == dev and ids.device == dev
            and w.codes.device == dev
            and A.is_contiguous() and B.is_contiguous() and scale.is_contiguous() and ids.is_contiguous()):
        _need(A, "A", bf, (count, r, w.k), dev)
        _need(B, "B", bf, (count, w.n, r), dev)
        _need(scale, "scale", torch.float32, (count,), dev)
        _need(ids, "ids", torch.int32, (m,), dev)
        _need_weight(w, dev)
    return AdapterSetC(A.data_ptr(), B.data_ptr(), scale.data_ptr(), count, r), count, r


def _multi_workspace(op, m, n, k, r, count, ws, device, stream):
    if ws is None:
        need = qlora_multi_workspace_bytes(op, m, n, k, r, count)
        # Sizes the library refuses have no workspace; the call reports them.
        ws = _empty(need if need < 1 << 62 else 0, torch.uint8, device, stream)
    _need_ws(ws, device)
    return ws, ws.numel() * ws.element_size()


def qlora_linear_fwd_multi(X: torch.Tensor, w: NF4Weight, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                           ids: torch.Tensor, out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """Y[i] = bf16(X[i] . W^T + bf16(s_a X[i] A_a^T) . B_a^T), a = ids[i]; an
    id outside [0, count) means no adapter.  X bf16 [m x k], A [count x r x k],
    B [count x n x r], scale fp32 [count], ids int32 [m].  The first m*r*2
    bytes of `ws` hold T afterwards, which qlora_linear_bwd_multi takes (it may
    have the same `ws`)."""
    m, dev = X.shape[0], X.device
    out = _out(out, (m, w.n), dev, stream)
    bf = torch.bfloat16
    if not (X.dtype is bf and out.dtype is bf and X.shape == (m, w.k) and out.shape == (m, w.n) and out.device == dev
            and X.is_contiguous() and out.is_contiguous()):
        _need(X, "X", bf, (m, w.k), dev)
        _need(out, "out", bf, (m, w.n), dev)
    set_c, count, r = _adapter_set(A, B, scale, ids, m, w, dev)
    ws, ws_bytes = _multi_workspace(QLORA_OP_FWD, m, w.n, w.k, r, count, ws, dev, stream)
    w_c = w.c_struct()
    _check("qlora_linear_fwd_multi",
           lib().qlora_linear_fwd_multi(X.data_ptr(), m, ctypes.byref(w_c), ctypes.byref(set_c), ids.data_ptr(),
                                        out.data_ptr(), ws.data_ptr(), ws_bytes, _stream_on(dev, stream)))
    return out


def qlora_linear_bwd_multi(dY: torch.Tensor, X, w: NF4Weight, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                           ids: torch.Tensor, T: Optional[torch.Tensor] = None, dX: Optional[torch.Tensor] = None,
                           dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None, want_dx: bool = True,
                           ws: Optional[torch.Tensor] = None, stream=None):
    """(dX or None, dA [count x r x k], dB [count x n x r]) of the layer whose
    rows have their own adapters (see qlora_linear_fwd_multi).  X is the bf16
    input or its Act8 checkpoint; T the forward's, required with a checkpoint."""
    m, n, k, dev, bf = dY.shape[0], w.n, w.k, dY.device, torch.bfloat16
    set_c, count, r = _adapter_set(A, B, scale, ids, m, w, dev)
    if dX is not None or want_dx:
        dX = _out(dX, (m, k), dev, stream)
    dA, dB = _out(dA, (count, r, k), dev, stream), _out(dB, (count, n, r), dev, stream)
    act = X if isinstance(X, Act8) else None
    if act is not None:
        _need_act8(act, m, k, dev)
        X = None
    for t, name, shape in ((dY, "dY", (m, n)), (X, "X", (m, k)), (T, "T", (m, r)), (dX, "dX", (m, k)),
                           (dA, "dA", (count, r, k)), (dB, "dB", (count, n, r))):
        _need(t, name, bf, shape, dev)
    ws, ws_bytes = _multi_workspace(QLORA_OP_LORA_BWD, m, n, k, r, count, ws, dev, stream)
    w_c = w.c_struct()
    a_c = ctypes.byref(act.c_struct()) if act is not None else None
    _check("qlora_linear_bwd_multi",
           lib().qlora_linear_bwd_multi(dY.data_ptr(), _ptr(X), a_c, _ptr(T), m, ctypes.byref(w_c),
                                        ctypes.byref(set_c), ids.data_ptr(), _ptr(dX), dA.data_ptr(), dB.data_ptr(),
                                        ws.data_ptr(), ws_bytes, _stream_on(dev, stream)))
    return dX, dA, dB


def qlora_selftest_bounded_wait(limit_ns: int, expired: Optional[torch.Tensor] = None, stream=None) -> None:
    """Launch the bounded-wait self-test (a wait on a barrier nothing arrives
    at, given up after limit_ns); `expired` is an int32 [1] device tensor that
    receives 1 when the wait ran out."""
    _need_cuda(expired)
    _check("qlora_selftest_bounded_wait",
           lib().qlora_selftest_bounded_wait(int(limit_ns), _ptr(expired), _stream(stream)))


def qlora_selftest_div255(first_bits: int, count: int, mismatches: torch.Tensor, stream=None) -> None:
    """Add to the int64 [1] device tensor `mismatches` the number of fp32 bit
    patterns in [first_bits, first_bits + count) whose library fp32(s / 255)
    differs from IEEE division."""
    _need_cuda(mismatches)
    _check("qlora_selftest_div255",
           lib().qlora_selftest_div255(int(first_bits), int(count), mismatches.data_ptr(), _stream(stream)))
