"""Thin Python binding of librsq.so (include/rsq.h): argument marshalling only.

Every step of the path runs in the library's CUDA kernels.  PyTorch supplies
device memory and the current CUDA stream.  There is no CPU fallback: if the
library is missing, importing this module raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librsq.so")

RSQ_F32, RSQ_BF16, RSQ_F16 = 0, 1, 2

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
        "or `python w3a3_quantization_online_b200/build.py` (the CUDA path has no fallback)")

_lib = ctypes.CDLL(LIB_PATH)
_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_lib.rsq_residual_align.argtypes = [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp]
_lib.rsq_residual_align.restype = _i32
_lib.rsq_align_norm_quant.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _f32, _i32, _vp]
_lib.rsq_align_norm_quant.restype = _i32
_lib.rht_quant.argtypes = [_vp, _vp, _i32, _vp, _vp, _i64, _i32, _i32, _i32, _vp]
_lib.rht_quant.restype = _i32
_lib.rht_quant_silu_gate.argtypes = [_vp, _vp, _vp, _i32, _vp, _vp, _i64, _i32, _i32, _i32, _vp]
_lib.rht_quant_silu_gate.restype = _i32
_lib.rht_heads.argtypes = [_vp, _vp, _i32, _vp, _i64, _i32, _i32, _vp]
_lib.rht_heads.restype = _i32
_lib.rht_heads_quant.argtypes = [_vp, _vp, _i32, _vp, _vp, _i64, _i32, _i32, _i32, _vp]
_lib.rht_heads_quant.restype = _i32
_lib.rht_head_mix_quant.argtypes = [_vp, _vp, _i32, _vp, _vp, _i64, _i32, _i32, _i32, _vp]
_lib.rht_head_mix_quant.restype = _i32
_lib.kron_affine_quant.argtypes = [_vp, _vp, _vp, _i32, _i32, _vp, _vp, _i64, _i32, _i32, _vp]
_lib.kron_affine_quant.restype = _i32
_lib.w4a4_gemm.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp]
_lib.w4a4_gemm.restype = _i32
_lib.w4a4_prepare_weights.argtypes = [_vp, _i32, _i32, _vp, _vp]
_lib.w4a4_prepare_weights.restype = _i32
_lib.w4a4_gemm_s8w.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp]
_lib.w4a4_gemm_s8w.restype = _i32
_lib.kv8_plan.argtypes = [_vp, _vp, _i32, _vp, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp]
_lib.kv8_plan.restype = _i32
_lib.kv8_plan_i64.argtypes = _lib.kv8_plan.argtypes
_lib.kv8_plan_i64.restype = _i32
_lib.kv8_append.argtypes = [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i64, _i32, _vp]
_lib.kv8_append.restype = _i32
_lib.kv8_attention.argtypes = [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _f32, _vp, _i64, _i32, _i32, _i32,
                               _i32, _i64, _i32, _vp, ctypes.c_uint64, _vp]
_lib.kv8_attention.restype = _i32
_lib.kv8_attention_i64.argtypes = _lib.kv8_attention.argtypes
_lib.kv8_attention_i64.restype = _i32
_lib.kv8_attention_workspace_bytes.argtypes = [_i64, _i32, _i32, _i32, _i32]
_lib.kv8_attention_workspace_bytes.restype = ctypes.c_uint64
_lib.w4_matvec.argtypes = [_vp, _i64, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _vp]
_lib.w4_matvec.restype = _i32
_lib.rsq_qm_build.argtypes = [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, ctypes.c_uint64, _vp]
_lib.rsq_qm_build.restype = _i32
_lib.rsq_qm_workspace_bytes.argtypes = [_i32, _i32]
_lib.rsq_qm_build_fixed_scratch.argtypes = [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp]
_lib.rsq_qm_build_fixed_scratch.restype = _i32
_lib.rsq_qm_workspace_bytes.restype = ctypes.c_uint64
_lib.rsq_status_string.argtypes = [_i32]
_lib.rsq_status_string.restype = ctypes.c_char_p
_lib.rsq_last_cuda_error.argtypes = []
_lib.rsq_last_cuda_error.restype = _i32
_lib.rsq_launch_count.argtypes = []
_lib.rsq_launch_count.restype = ctypes.c_uint64
_lib.rsq_select_align_kernel.argtypes = [_i32]
_lib.rsq_select_align_kernel.restype = _i32
_lib.rsq_select_rht_kernel.argtypes = [_i32]
_lib.rsq_select_rht_kernel.restype = _i32
_lib.rsq_device_status.argtypes = [_vp, ctypes.POINTER(_i32)]
_lib.rsq_device_status.restype = _i32
_lib.rsq_selftest_wait_timeout.argtypes = [_i32, _vp]
_lib.rsq_selftest_wait_timeout.restype = _i32

EXPORTED = ("rsq_residual_align", "rsq_align_norm_quant", "rht_quant", "rht_quant_silu_gate", "rht_heads",
            "rht_heads_quant", "rht_head_mix_quant", "kron_affine_quant", "w4a4_gemm", "w4a4_prepare_weights", "w4a4_gemm_s8w",
            "kv8_plan", "kv8_plan_i64", "kv8_append", "kv8_attention", "kv8_attention_i64", "kv8_attention_workspace_bytes", "w4_matvec",
            "rsq_qm_build", "rsq_qm_workspace_bytes",
            "rsq_qm_build_fixed_scratch",
            "rsq_status_string",
            "rsq_last_cuda_error", "rsq_launch_count", "rsq_select_align_kernel", "rsq_select_rht_kernel", "rsq_device_status",
            "rsq_selftest_wait_timeout")

ALIGN_AUTO, ALIGN_GENERIC, ALIGN_TENSOR_CORE, ALIGN_DECODE = 0, 1, 2, 4
RHT_AUTO, RHT_GENERIC, RHT_TENSOR_CORE, RHT_KRONECKER = 0, 1, 3, 4


class RsqError(RuntimeError):
    def __init__(self, status: int):
        msg = _lib.rsq_status_string(status).decode()
        if status == 8:
            msg += f" (cudaError {int(_lib.rsq_last_cuda_error())})"
        super().__init__(msg)
        self.status = status


def library() -> ctypes.CDLL:
    return _lib


def launch_count() -> int:
    return int(_lib.rsq_launch_count())


def select_align_kernel(which: int) -> int:
    """0 auto, 1 CUDA-core, 2 tensor-core cluster kernel (one 128-row tile per CTA), 4 decode kernel;
    returns the previous setting."""
    prev = int(_lib.rsq_select_align_kernel(int(which)))
    if prev < 0:
        raise ValueError(which)
    return prev


def select_rht_kernel(which: int) -> int:
    """0 auto, 1 radix-16 SMEM kernel, 3 tensor-core kernel, 4 Kronecker kernel; returns the previous setting."""
    prev = int(_lib.rsq_select_rht_kernel(int(which)))
    if prev < 0:
        raise ValueError(which)
    return prev


def device_status(stream=None) -> int:
    """Take (and clear) the device status word on the stream, after the work
    queued on it; returns it (0 = healthy).  The word is per device and shared
    by all streams."""
    out = _i32(0)
    _check(_lib.rsq_device_status(_stream(stream), ctypes.byref(out)))
    return int(out.value)


def selftest_wait_timeout(limit_ms: int = 20, stream=None) -> None:
    """Enqueue the bounded-wait self test (a wait that runs out after limit_ms
    and sets the timeout bit of the device status word)."""
    _check(_lib.rsq_selftest_wait_timeout(int(limit_ms), _stream(stream)))


def status_string(status: int) -> str:
    return _lib.rsq_status_string(status).decode()


def _check(status: int) -> None:
    if status != 0:
        raise RsqError(status)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return RSQ_F32
    if t.dtype == torch.bfloat16:
        return RSQ_BF16
    raise TypeError(f"activations must be float32 or bfloat16, got {t.dtype}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _need(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def rsq_residual_align(x: torch.Tensor, Q: torch.Tensor, M: torch.Tensor,
                       x_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x_out = x + Q (M (Q^T x)) per row of the T x D activations x (in place if x_out is x)."""
    _need(x, "x"); _need(Q, "Q", torch.float32); _need(M, "M", torch.float32)
    T, D = x.shape
    r = Q.shape[1]
    if x_out is None:
        x_out = torch.empty_like(x)
    _need(x_out, "x_out", x.dtype)
    _check(_lib.rsq_residual_align(_ptr(x), _ptr(Q), _ptr(M), _ptr(x_out), T, D, r,
                                   _dtype_code(x), _stream(stream)))
    return x_out


def rsq_align_norm_quant(x: torch.Tensor, Q: torch.Tensor, M: torch.Tensor,
                         x_out: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
                         scales: Optional[torch.Tensor] = None, bits: int = 4, eps: float = 1e-5,
                         stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Alignment -> weight-free RMSNorm -> per-token symmetric INT{bits} codes.

    Returns (x_out, codes uint8 T x D*bits/8, scales float32 T)."""
    _need(x, "x"); _need(Q, "Q", torch.float32); _need(M, "M", torch.float32)
    T, D = x.shape
    r = Q.shape[1]
    if x_out is None:
        x_out = torch.empty_like(x)
    if codes is None:
        codes = torch.empty((T, D * bits // 8), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((T,), dtype=torch.float32, device=x.device)
    _need(x_out, "x_out", x.dtype); _need(codes, "codes", torch.uint8); _need(scales, "scales", torch.float32)
    _check(_lib.rsq_align_norm_quant(_ptr(x), _ptr(Q), _ptr(M), _ptr(x_out), _ptr(codes), _ptr(scales),
                                     T, D, r, bits, float(eps), _dtype_code(x), _stream(stream)))
    return x_out, codes, scales


def rht_quant(x: torch.Tensor, signs: torch.Tensor, m: int = 1, codes: Optional[torch.Tensor] = None,
              scales: Optional[torch.Tensor] = None, bits: int = 4,
              stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Randomised Hadamard H_d diag(signs) x / sqrt(d) -> per-token symmetric INT{bits} codes.

    Returns (codes uint8 T x d*bits/8, scales float32 T)."""
    _need(x, "x"); _need(signs, "signs", torch.int8)
    T, d = x.shape
    if codes is None:
        codes = torch.empty((T, d * bits // 8), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((T,), dtype=torch.float32, device=x.device)
    _need(codes, "codes", torch.uint8); _need(scales, "scales", torch.float32)
    _check(_lib.rht_quant(_ptr(x), _ptr(signs), m, _ptr(codes), _ptr(scales), T, d, bits,
                          _dtype_code(x), _stream(stream)))
    return codes, scales


def rht_quant_silu_gate(a: torch.Tensor, b: torch.Tensor, signs: torch.Tensor, m: int = 1,
                        codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                        bits: int = 4, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """SiLU(a) * b -> randomised Hadamard H_d diag(signs) / sqrt(d) -> per-token INT{bits} codes.

    Returns (codes uint8 T x d*bits/8, scales float32 T)."""
    _need(a, "a"); _need(b, "b", a.dtype); _need(signs, "signs", torch.int8)
    T, d = a.shape
    if tuple(b.shape) != (T, d):
        raise ValueError(f"b has shape {tuple(b.shape)}, expected {(T, d)}")
    if codes is None:
        codes = torch.empty((T, d * bits // 8), dtype=torch.uint8, device=a.device)
    if scales is None:
        scales = torch.empty((T,), dtype=torch.float32, device=a.device)
    _need(codes, "codes", torch.uint8); _need(scales, "scales", torch.float32)
    _check(_lib.rht_quant_silu_gate(_ptr(a), _ptr(b), _ptr(signs), m, _ptr(codes), _ptr(scales), T, d, bits,
                                    _dtype_code(a), _stream(stream)))
    return codes, scales


def _signs_ptr(signs: Optional[torch.Tensor]) -> Optional[int]:
    if signs is None:
        return None
    _need(signs, "signs", torch.int8)
    return signs.data_ptr()


def rht_heads(x: torch.Tensor, signs: Optional[torch.Tensor], n_heads: int,
              x_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Per-head rotation (I (x) H_{d_h}) diag(signs) x / sqrt(d_h) of queries or keys (in place if x_out is x)."""
    _need(x, "x")
    T, d = x.shape
    if x_out is None:
        x_out = torch.empty_like(x)
    _need(x_out, "x_out", x.dtype)
    _check(_lib.rht_heads(_ptr(x), _signs_ptr(signs), n_heads, _ptr(x_out), T, d, _dtype_code(x), _stream(stream)))
    return x_out


def rht_heads_quant(x: torch.Tensor, signs: Optional[torch.Tensor], n_heads: int, codes: Optional[torch.Tensor] = None,
                    scales: Optional[torch.Tensor] = None, bits: int = 4,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-head rotation, then per-(token, head) INT{bits} codes.  Returns (codes T x d*bits/8, scales T x n_heads)."""
    _need(x, "x")
    T, d = x.shape
    if codes is None:
        codes = torch.empty((T, d * bits // 8), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((T, n_heads), dtype=torch.float32, device=x.device)
    _need(codes, "codes", torch.uint8); _need(scales, "scales", torch.float32)
    _check(_lib.rht_heads_quant(_ptr(x), _signs_ptr(signs), n_heads, _ptr(codes), _ptr(scales), T, d, bits,
                                _dtype_code(x), _stream(stream)))
    return codes, scales


def rht_head_mix_quant(x: torch.Tensor, signs: Optional[torch.Tensor], n_heads: int,
                       codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None, bits: int = 4,
                       stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Head mixing (H_{n_h} (x) I) diag(signs) x / sqrt(n_h), then per-token INT{bits} codes."""
    _need(x, "x")
    T, d = x.shape
    if codes is None:
        codes = torch.empty((T, d * bits // 8), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((T,), dtype=torch.float32, device=x.device)
    _need(codes, "codes", torch.uint8); _need(scales, "scales", torch.float32)
    _check(_lib.rht_head_mix_quant(_ptr(x), _signs_ptr(signs), n_heads, _ptr(codes), _ptr(scales), T, d, bits,
                                   _dtype_code(x), _stream(stream)))
    return codes, scales


def kron_affine_quant(x: torch.Tensor, P1: torch.Tensor, P2: torch.Tensor,
                      codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None, bits: int = 4,
                      stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """FlatQuant's Kronecker affine transform vec(P1^T X P2) of each row, then per-token INT{bits} codes."""
    _need(x, "x")
    _need(P1, "P1", torch.float32); _need(P2, "P2", torch.float32)
    T, d = x.shape
    n1, n2 = P1.shape[0], P2.shape[0]
    if P1.shape != (n1, n1) or P2.shape != (n2, n2) or n1 * n2 != d:
        raise ValueError(f"P1 {tuple(P1.shape)} and P2 {tuple(P2.shape)} do not factor a row of {d}")
    if codes is None:
        codes = torch.empty((T, d * bits // 8), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((T,), dtype=torch.float32, device=x.device)
    _need(codes, "codes", torch.uint8); _need(scales, "scales", torch.float32)
    _check(_lib.kron_affine_quant(_ptr(x), _ptr(P1), _ptr(P2), n1, n2, _ptr(codes), _ptr(scales), T, bits,
                                  _dtype_code(x), _stream(stream)))
    return codes, scales


def w4a4_gemm(codes_a: torch.Tensor, scales_a: torch.Tensor, codes_w: torch.Tensor, scales_w: torch.Tensor,
              y: Optional[torch.Tensor] = None, acc: Optional[torch.Tensor] = None, out_dtype=torch.float16,
              stream=None) -> torch.Tensor:
    """Y = (INT4 codes_a @ INT4 codes_w^T) * scales_a[:, None] * scales_w[None, :] in fp16 / bf16.

    codes_a: T x K/2 uint8, codes_w: N x K/2 uint8 (packed INT4); acc (optional) receives the int32 products."""
    _need(codes_a, "codes_a", torch.uint8); _need(codes_w, "codes_w", torch.uint8)
    _need(scales_a, "scales_a", torch.float32); _need(scales_w, "scales_w", torch.float32)
    T, kb = codes_a.shape
    N = codes_w.shape[0]
    if codes_w.shape[1] != kb:
        raise ValueError("codes_a and codes_w disagree on K")
    if out_dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("out_dtype must be float16 or bfloat16")
    if y is None:
        y = torch.empty((T, N), dtype=out_dtype, device=codes_a.device)
    _need(y, "y", out_dtype)
    if acc is not None:
        _need(acc, "acc", torch.int32)
    code = RSQ_F16 if out_dtype == torch.float16 else RSQ_BF16
    _check(_lib.w4a4_gemm(_ptr(codes_a), _ptr(scales_a), _ptr(codes_w), _ptr(scales_w), _ptr(y), _ptr(acc), T, N,
                          2 * kb, code, _stream(stream)))
    return y


def w4a4_prepare_weights(codes_w: torch.Tensor, w_s8: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The packed INT4 weight codes (N x K/2 uint8) unpacked once to int8 (N x K) for w4a4_gemm_s8w."""
    _need(codes_w, "codes_w", torch.uint8)
    N, kb = codes_w.shape
    if w_s8 is None:
        w_s8 = torch.empty((N, 2 * kb), dtype=torch.int8, device=codes_w.device)
    _need(w_s8, "w_s8", torch.int8)
    if tuple(w_s8.shape) != (N, 2 * kb):
        raise ValueError("w_s8 must be N x K")
    _check(_lib.w4a4_prepare_weights(_ptr(codes_w), N, 2 * kb, _ptr(w_s8), _stream(stream)))
    return w_s8


def w4a4_gemm_s8w(codes_a: torch.Tensor, scales_a: torch.Tensor, w_s8: torch.Tensor, scales_w: torch.Tensor,
                  y: Optional[torch.Tensor] = None, acc: Optional[torch.Tensor] = None, out_dtype=torch.float16,
                  stream=None) -> torch.Tensor:
    """w4a4_gemm with the weights prepared by w4a4_prepare_weights (N x K int8)."""
    _need(codes_a, "codes_a", torch.uint8); _need(w_s8, "w_s8", torch.int8)
    _need(scales_a, "scales_a", torch.float32); _need(scales_w, "scales_w", torch.float32)
    T, kb = codes_a.shape
    N = w_s8.shape[0]
    if w_s8.shape[1] != 2 * kb:
        raise ValueError("codes_a and w_s8 disagree on K")
    if out_dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("out_dtype must be float16 or bfloat16")
    if y is None:
        y = torch.empty((T, N), dtype=out_dtype, device=codes_a.device)
    _need(y, "y", out_dtype)
    if acc is not None:
        _need(acc, "acc", torch.int32)
    code = RSQ_F16 if out_dtype == torch.float16 else RSQ_BF16
    _check(_lib.w4a4_gemm_s8w(_ptr(codes_a), _ptr(scales_a), _ptr(w_s8), _ptr(scales_w), _ptr(y), _ptr(acc), T, N,
                              2 * kb, code, _stream(stream)))
    return y


def _enter(device_index: int, stream):
    """What a call on tensors of this device has to make current around it, where that is not so already: their
    device (the library works on the current one) and, where the caller names a stream, that stream, so that what
    the call allocates belongs to the stream it runs on."""
    if stream is None:
        return torch.cuda.device(device_index)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=torch.device("cuda", device_index))
    if stream.device_index != device_index:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{device_index}")
    return torch.cuda.stream(stream)


# The current stream's handle and the current device, by torch's own short cuts where this torch has them: a few
# microseconds less per call than the public ones.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device_index: torch.cuda.current_stream(device_index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _lists_ok(device_index: int, dtype, *tensors: torch.Tensor) -> bool:
    """All contiguous, of that type, on that device."""
    for t in tensors:
        if t.dtype is not dtype or t.get_device() != device_index or not t.is_contiguous():
            return False
    return True


def _refuse(device_index: int, dtype, **tensors: torch.Tensor) -> None:
    """Says what _lists_ok found wrong."""
    for name, t in tensors.items():
        _need(t, name, dtype)
        if t.get_device() != device_index:
            raise ValueError(f"{name} is on {t.device}, the call's first tensor on cuda:{device_index}")


def _rows(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """(rows, width, elements from row to row) of a CUDA matrix whose rows are contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    n, width = t.shape
    ld, step = t.stride()
    if step != 1 and width > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return n, width, ld if n > 1 else width


def _cache(device_index: int, k_cache, k_scale, v_cache, v_scale):
    """(n_blocks, n_kv, block_size, d_h) of a cache."""
    if not (k_cache.dtype is torch.int8 and v_cache.dtype is torch.int8 and k_scale.dtype is torch.float32 and
            v_scale.dtype is torch.float32 and k_cache.is_contiguous() and v_cache.is_contiguous() and
            k_scale.is_contiguous() and v_scale.is_contiguous() and
            k_cache.get_device() == v_cache.get_device() == k_scale.get_device() == v_scale.get_device() == device_index):
        _refuse(device_index, torch.int8, k_cache=k_cache, v_cache=v_cache)
        _refuse(device_index, torch.float32, k_scale=k_scale, v_scale=v_scale)
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be n_blocks x n_kv x block_size x d_h, both alike")
    if k_scale.shape != shape[:2] or v_scale.shape != shape[:2]:
        raise ValueError("k_scale and v_scale must be n_blocks x n_kv")
    return shape


def _table_ok(device_index: int, block_table: torch.Tensor) -> bool:
    """A block table of int32 or int64 ids."""
    return _lists_ok(device_index, torch.int64 if block_table.dtype is torch.int64 else torch.int32, block_table)


def _refuse_table(device_index: int, block_table: torch.Tensor) -> None:
    """Says what _table_ok found wrong."""
    if block_table.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"block_table must be int32 or int64, got {block_table.dtype}")
    _refuse(device_index, block_table.dtype, block_table=block_table)


def kv8_plan(ctx_len: torch.Tensor, new_len: torch.Tensor, block_table: torch.Tensor, free_blocks: torch.Tensor,
             cursor: torch.Tensor, T: int, block_size: int,
             stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Block tables and slots of a batch of new tokens, on the GPU, from the requests' lengths.

    ctx_len, new_len: int32 B; block_table: int32 or int64 B x max_blocks, completed in place with
    ids free_blocks[cursor], free_blocks[cursor + 1], ... (int32; cursor: int32, one element); T:
    rows of the (padded) batch.  Returns (cu_new int32 B + 1, seq_len int32 B, positions int32 T,
    slots int64 T, cursor_out int32 1); padding rows get position and slot -1."""
    d = ctx_len.get_device()
    if d < 0 or not (_lists_ok(d, torch.int32, ctx_len, new_len, free_blocks, cursor) and _table_ok(d, block_table)):
        _refuse(d, torch.int32, ctx_len=ctx_len, new_len=new_len, free_blocks=free_blocks, cursor=cursor)
        _refuse_table(d, block_table)
    B = ctx_len.numel()
    if new_len.numel() != B or block_table.dim() != 2 or block_table.shape[0] != B or cursor.numel() != 1:
        raise ValueError("new_len must have B elements, block_table B rows and cursor one element")
    if stream is not None or _current_device() != d:
        with _enter(d, stream):
            return kv8_plan(ctx_len, new_len, block_table, free_blocks, cursor, T, block_size)
    # one allocation for the int32 results
    cu_new, seq_len, positions, cursor_out = ctx_len.new_empty(2 * B + 2 + T).split_with_sizes((B + 1, B, T, 1))
    slots = ctx_len.new_empty(T, dtype=torch.int64)
    call = _lib.kv8_plan_i64 if block_table.dtype is torch.int64 else _lib.kv8_plan
    _check(call(ctx_len.data_ptr(), new_len.data_ptr(), B, block_table.data_ptr(), block_table.shape[1], block_size,
                free_blocks.data_ptr(), free_blocks.numel(), cursor.data_ptr(), cursor_out.data_ptr(), cu_new.data_ptr(),
                seq_len.data_ptr(), positions.data_ptr(), slots.data_ptr(), T, _raw_stream(d)))
    return cu_new, seq_len, positions, slots, cursor_out


def kv8_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor, k_scale: torch.Tensor,
               v_cache: torch.Tensor, v_scale: torch.Tensor, stream=None) -> None:
    """Quantise keys and values (T x n_kv*d_h, rows may be strided) into the paged 8-bit cache, in place.

    slots: int64 T (negative: skipped); caches int8 n_blocks x n_kv x block_size x d_h, scales
    float32 n_blocks x n_kv."""
    T, width, ldk = _rows(k, "k")
    Tv, width_v, ldv = _rows(v, "v")
    d = k.get_device()
    n_blocks, n_kv, block_size, d_h = _cache(d, k_cache, k_scale, v_cache, v_scale)
    if not _lists_ok(d, torch.int64, slots):
        _refuse(d, torch.int64, slots=slots)
    if v.dtype != k.dtype or v.get_device() != d:
        raise TypeError(f"v must be {k.dtype} on {k.device}, got {v.dtype} on {v.device}")
    if width != n_kv * d_h or width_v != width or Tv != T or slots.numel() != T:
        raise ValueError(f"k and v must be T x {n_kv * d_h} and slots T")
    if stream is not None or _current_device() != d:
        with _enter(d, stream):
            return kv8_append(k, v, slots, k_cache, k_scale, v_cache, v_scale)
    _check(_lib.kv8_append(k.data_ptr(), ldk, v.data_ptr(), ldv, slots.data_ptr(), k_cache.data_ptr(),
                           k_scale.data_ptr(), v_cache.data_ptr(), v_scale.data_ptr(), T, n_kv, d_h, block_size,
                           n_blocks, _dtype_code(k), _raw_stream(d)))


def kv8_attention_workspace_bytes(T: int, B: int, n_heads: int, n_kv: int, d_h: int) -> int:
    return int(_lib.kv8_attention_workspace_bytes(T, B, n_heads, n_kv, d_h))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(device_index: int, T: int, B: int, n_heads: int, n_kv: int, d_h: int) -> int:
    need = kv8_attention_workspace_bytes(T, B, n_heads, n_kv, d_h)
    if need == 0:
        raise RsqError(2)
    return need


def kv8_attention(q: torch.Tensor, k_cache: torch.Tensor, k_scale: torch.Tensor, v_cache: torch.Tensor,
                  v_scale: torch.Tensor, block_table: torch.Tensor, seq_len: torch.Tensor, cu_new: torch.Tensor,
                  sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention of the new tokens' queries (T x n_heads*d_h) over the paged 8-bit cache.

    block_table: int32 or int64 B x max_blocks, seq_len: int32 B (the new tokens counted), cu_new: int32
    B + 1.  sm_scale defaults to 1 / sqrt(d_h).  Rows behind cu_new[B] of out keep their contents.
    workspace: a uint8 CUDA tensor of at least kv8_attention_workspace_bytes(...) (allocated here
    when None).  Returns out (T x n_heads*d_h)."""
    T, width, ldq = _rows(q, "q")
    d = q.get_device()
    n_blocks, n_kv, block_size, d_h = _cache(d, k_cache, k_scale, v_cache, v_scale)
    if not (_lists_ok(d, torch.int32, seq_len, cu_new) and _table_ok(d, block_table)):
        _refuse(d, torch.int32, seq_len=seq_len, cu_new=cu_new)
        _refuse_table(d, block_table)
    B = seq_len.numel()
    if d_h == 0 or width % d_h or block_table.dim() != 2 or block_table.shape[0] != B or cu_new.numel() != B + 1:
        raise ValueError("q must have whole heads, block_table B rows and cu_new B + 1 elements")
    if stream is not None or _current_device() != d:
        with _enter(d, stream):
            return kv8_attention(q, k_cache, k_scale, v_cache, v_scale, block_table, seq_len, cu_new, sm_scale, out,
                                 workspace)
    n_heads = width // d_h
    if out is None:
        out = torch.empty_like(q) if ldq == width else q.new_empty((T, width))
    elif out.dtype != q.dtype or out.shape != q.shape or not _lists_ok(d, q.dtype, out):
        _refuse(d, q.dtype, out=out)
        raise ValueError("out must have q's shape")
    if workspace is None:
        workspace = k_cache.new_empty(_workspace_bytes(d, T, B, n_heads, n_kv, d_h))
    elif not _lists_ok(d, torch.uint8, workspace):
        _refuse(d, torch.uint8, workspace=workspace)
    call = _lib.kv8_attention_i64 if block_table.dtype is torch.int64 else _lib.kv8_attention
    _check(call(q.data_ptr(), ldq, k_cache.data_ptr(), k_scale.data_ptr(), v_cache.data_ptr(), v_scale.data_ptr(),
                block_table.data_ptr(), block_table.shape[1], seq_len.data_ptr(), cu_new.data_ptr(), B,
                d_h ** -0.5 if sm_scale is None else sm_scale, out.data_ptr(), T, n_heads, n_kv, d_h, block_size,
                n_blocks, _dtype_code(q), workspace.data_ptr(), workspace.numel(), _raw_stream(d)))
    return out


def w4_matvec(x: torch.Tensor, codes_w: torch.Tensor, scales_w: torch.Tensor, y: Optional[torch.Tensor] = None,
              out_dtype=None, stream=None) -> torch.Tensor:
    """y = x W^T for a few rows x (T x K, rows may be strided), W[n][k] = codes_w[n][k] * scales_w[n][k / group].

    codes_w: N x K/2 uint8 (packed INT4), scales_w: N x K/group float32; out_dtype defaults to x's."""
    T, K, ldx = _rows(x, "x")
    d = x.get_device()
    if not (codes_w.dtype is torch.uint8 and scales_w.dtype is torch.float32 and codes_w.is_contiguous() and
            scales_w.is_contiguous() and codes_w.get_device() == scales_w.get_device() == d):
        _refuse(d, torch.uint8, codes_w=codes_w)
        _refuse(d, torch.float32, scales_w=scales_w)
    if codes_w.dim() != 2 or scales_w.dim() != 2:
        raise ValueError("codes_w and scales_w must be matrices")
    N, half = codes_w.shape
    rows, groups = scales_w.shape
    if 2 * half != K:
        raise ValueError("codes_w must be N x K/2")
    if rows != N or groups == 0 or K % groups:
        raise ValueError("scales_w must be N x K/group")
    dtype = x.dtype
    if out_dtype is None:
        out_dtype = dtype if y is None else y.dtype
    code = _OUT_CODES.get(out_dtype)
    if code is None:
        raise TypeError("out_dtype must be float32, bfloat16 or float16")
    if stream is not None or _current_device() != d:
        with _enter(d, stream):
            return w4_matvec(x, codes_w, scales_w, y, out_dtype)
    if y is None:
        y = x.new_empty((T, N)) if out_dtype is dtype else x.new_empty((T, N), dtype=out_dtype)
    elif y.shape != (T, N) or not _lists_ok(d, out_dtype, y):
        _refuse(d, out_dtype, y=y)
        raise ValueError("y must be T x N")
    _check(_lib.w4_matvec(x.data_ptr(), ldx, codes_w.data_ptr(), scales_w.data_ptr(), y.data_ptr(), T, N, K,
                          K // groups, _dtype_code(x), code, _raw_stream(d)))
    return y


_OUT_CODES = {torch.float32: RSQ_F32, torch.bfloat16: RSQ_BF16, torch.float16: RSQ_F16}


def qm_workspace_bytes(D: int, r: int) -> int:
    return int(_lib.rsq_qm_workspace_bytes(D, r))


def qm_build(R_in: torch.Tensor, R_out: torch.Tensor, r: int, iters: int = 16,
             workspace: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Offline (Q, M) of the alignment from the rotations on both sides of a residual connection.

    Returns (Q D x r float32, M r x r float32).  workspace: a uint8 CUDA tensor of at
    least qm_workspace_bytes(D, r) bytes (allocated here when None)."""
    _need(R_in, "R_in", torch.float32); _need(R_out, "R_out", torch.float32)
    D = R_in.shape[0]
    need = qm_workspace_bytes(D, r)
    if need == 0:
        raise RsqError(2)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=R_in.device)
    _need(workspace, "workspace", torch.uint8)
    Q = torch.empty((D, r), dtype=torch.float32, device=R_in.device)
    M = torch.empty((r, r), dtype=torch.float32, device=R_in.device)
    _check(_lib.rsq_qm_build(_ptr(R_in), _ptr(R_out), D, r, iters, _ptr(Q), _ptr(M), _ptr(workspace),
                             workspace.numel(), _stream(stream)))
    return Q, M


def qm_build_fixed_scratch(R_in: torch.Tensor, R_out: torch.Tensor, r: int, iters: int = 16,
                           stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """qm_build on the library's own fixed scratch array (no workspace argument).

    Shapes whose workspace exceeds the array are rejected; calls whose work
    overlaps on the GPU share the array and must be serialised."""
    _need(R_in, "R_in", torch.float32); _need(R_out, "R_out", torch.float32)
    D = R_in.shape[0]
    Q = torch.empty((D, r), dtype=torch.float32, device=R_in.device)
    M = torch.empty((r, r), dtype=torch.float32, device=R_in.device)
    _check(_lib.rsq_qm_build_fixed_scratch(_ptr(R_in), _ptr(R_out), D, r, iters, _ptr(Q), _ptr(M), _stream(stream)))
    return Q, M
