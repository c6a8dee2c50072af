"""ctypes binding of libfp8q.so (the C ABI in include/fp8q.h).

Two layers, both argument marshalling only:

* ``fp8q_*`` functions with the C names and C argument lists (device pointers
  as Python ints, ``stream`` as an int handle or None);
* tensor helpers (``quantize_act``, ``quantize_weight``, ``requant_transpose``,
  ``gemm``, ``grouped_gemm``; ``layernorm``, ``swiglu_quantize``, their backward
  passes and ``moe_decode``; ``grouped_quantize_act``,
  ``grouped_requant_transpose``, ``grouped_wgrad`` and ``adamw``) that take
  torch tensors on the HIP device, allocate outputs and workspaces with torch,
  derive leading dimensions from strides and enqueue on torch's current stream.

Every computation runs in the library's HIP kernels.  If the library is not
built, importing this module raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional, Sequence, Tuple, Union

import torch
from torch.autograd.graph import increment_version

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8q.so")

FP8Q_OK = 0
FP8Q_EINVAL = 1
FP8Q_ESHAPE = 2
FP8Q_EALIGN = 3
FP8Q_EUNSUPPORTED = 4
FP8Q_EHIP = 5

FP8Q_F32 = 0
FP8Q_BF16 = 1
FP8Q_TILE_1x128 = 0
FP8Q_TILE_128x1 = 1
FP8Q_BSCALE_BLOCK128 = 0
FP8Q_BSCALE_ROW = 1
FP8Q_GEMM_MMA_FP8 = 1
FP8Q_GEMM_POW2_SCALES = 2
FP8Q_SCALE_FP32 = 0
FP8Q_SCALE_POW2 = 1
FP8Q_NORM_LAYER = 0
FP8Q_NORM_RMS = 1

EXPORTS = ("fp8q_quantize_act", "fp8q_quantize_weight", "fp8q_requant_transpose", "fp8q_gemm",
           "fp8q_grouped_gemm", "fp8q_gemm_ex", "fp8q_grouped_gemm_ex", "fp8q_quantize_act_ex",
           "fp8q_quantize_weight_ex", "fp8q_requant_transpose_ex", "fp8q_transpose_weight",
           "fp8q_gather_quantize_act", "fp8q_gemm_splitk", "fp8q_gemm_splitk_noalloc", "fp8q_clock_probe",
           "fp8q_layernorm", "fp8q_layernorm_backward", "fp8q_swiglu_quantize", "fp8q_swiglu_backward",
           "fp8q_swiglu_backward_quantize", "fp8q_moe_decode", "fp8q_grouped_quantize_act",
           "fp8q_grouped_requant_transpose", "fp8q_grouped_wgrad", "fp8q_adamw", "fp8q_grouped_padded_rows",
           "fp8q_grouped_wgrad_workspace", "fp8q_layernorm_backward_workspace", "fp8q_moe_decode_workspace",
           "fp8q_gemm_splitk_workspace", "fp8q_strerror", "fp8q_version")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() (hipcc, gfx950)")

_lib = ctypes.CDLL(LIB_PATH)
_p, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int

_lib.fp8q_quantize_act.argtypes = [_p, _i32, _i64, _i64, _i64, _i32, _p, _i64, _p, _i64, _p]
_lib.fp8q_quantize_weight.argtypes = [_p, _i32, _i64, _i64, _i64, _p, _i64, _p, _i64, _p]
_lib.fp8q_requant_transpose.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
_lib.fp8q_gemm.argtypes = [_p, _i64, _p, _i64, _p, _i64, _p, _i64, _i32, _i64, _i64, _i64, _p, _i32,
                           _i64, _i32, _p]
_lib.fp8q_grouped_gemm.argtypes = [_p, _i64, _p, _i64, _p, _i64, _i64, _p, _i64, _i64, _p, _i32, _i64,
                                   _i64, _i64, _p, _i32, _i64, _p]
_u32 = ctypes.c_uint
_lib.fp8q_gemm_ex.argtypes = _lib.fp8q_gemm.argtypes[:-1] + [_u32, _p]
_lib.fp8q_grouped_gemm_ex.argtypes = _lib.fp8q_grouped_gemm.argtypes[:-1] + [_u32, _p]
_lib.fp8q_quantize_act_ex.argtypes = _lib.fp8q_quantize_act.argtypes[:-1] + [_i32, _p]
_lib.fp8q_quantize_weight_ex.argtypes = _lib.fp8q_quantize_weight.argtypes[:-1] + [_i32, _p]
_lib.fp8q_requant_transpose_ex.argtypes = _lib.fp8q_requant_transpose.argtypes[:-1] + [_i32, _p]
_lib.fp8q_transpose_weight.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
_lib.fp8q_gather_quantize_act.argtypes = [_p, _i32, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _i32, _p]
_lib.fp8q_gemm_splitk.argtypes = _lib.fp8q_gemm.argtypes[:-1] + [_u32, _p, _i64, _p]
_lib.fp8q_gemm_splitk_noalloc.argtypes = _lib.fp8q_gemm.argtypes[:-1] + [_u32, _p]
_lib.fp8q_clock_probe.argtypes = [_p, _i64, _p]
_lib.fp8q_gemm_splitk_workspace.argtypes = [_i64, _i64, _i64]
_lib.fp8q_gemm_splitk_workspace.restype = _i64
_f32 = ctypes.c_float
_lib.fp8q_layernorm.argtypes = [_p, _i32, _i64, _i64, _i64, _p, _p, _i32, _f32, _i32, _p, _i32, _i64, _p, _i64, _p,
                                _i64, _i32, _p, _p, _p]
_lib.fp8q_layernorm_backward.argtypes = [_p, _i64, _p, _i64, _i32, _i64, _i64, _p, _i32, _p, _p, _i32, _p, _i64, _p,
                                         _i64, _p, _p, _i32, _p, _i64, _p]
_lib.fp8q_layernorm_backward_workspace.argtypes = [_i64, _i64]
_lib.fp8q_swiglu_quantize.argtypes = [_p, _p, _i32, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _i64, _p, _p, _i64,
                                      _i32, _p]
_lib.fp8q_swiglu_backward.argtypes = [_p, _p, _i64, _p, _p, _i64, _p, _i32, _i64, _i64, _i64, _p, _p, _i64, _p]
_lib.fp8q_swiglu_backward_quantize.argtypes = [_p, _p, _i64, _p, _p, _i64, _p, _i32, _i64, _i64, _i64, _p, _p, _i64,
                                               _p, _p, _i64, _p, _p, _i64, _p, _p, _i64, _p, _i64, _p, _i64, _i32, _p]
_lib.fp8q_moe_decode_workspace.argtypes = [_i64, _i64, _i64, _i32, _i32]
_lib.fp8q_moe_decode.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _i32, _i32, _i32, _i64, _p, _i64, _i64, _p, _i64,
                                 _i64, _p, _i64, _i64, _p, _i64, _i64, _p, _i32, _i64, _p, _i64, _p]
_lib.fp8q_grouped_padded_rows.argtypes = [_i64, _i32]
_lib.fp8q_grouped_quantize_act.argtypes = [_p, _i32, _i64, _i64, _i64, _p, _i32, _p, _i64, _p, _i64, _i32, _p]
_lib.fp8q_grouped_requant_transpose.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _p, _i32, _p, _i64, _p, _i64, _i32, _p]
_lib.fp8q_grouped_wgrad_workspace.argtypes = [_i64, _i32, _i64, _i64]
_lib.fp8q_grouped_wgrad.argtypes = [_p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i32, _i64, _i64, _i64, _p, _i32, _i64,
                                    _i64, _i32, _u32, _p, _i64, _p]
_f64 = ctypes.c_double


class fp8q_adamw_tensor(ctypes.Structure):
    _fields_ = [("n", _i64), ("p", _p), ("g", _p), ("m", _p), ("v", _p), ("sm", _p), ("sv", _p), ("N", _i64),
                ("K", _i64), ("q", _p), ("s", _p), ("qt", _p), ("st", _p)]


class fp8q_adamw_config(ctypes.Structure):
    _fields_ = [("lr", _f64), ("beta1", _f64), ("beta2", _f64), ("eps", _f64), ("weight_decay", _f64), ("step", _i64),
                ("lr_dev", _p), ("step_dev", _p), ("grad_scale", _p), ("seed", ctypes.c_uint32)]


_lib.fp8q_adamw.argtypes = [_p, _i32, _i32, _i32, _p, _i32, _p]
_lib.fp8q_strerror.argtypes = [_i32]
_lib.fp8q_strerror.restype = ctypes.c_char_p
_lib.fp8q_version.argtypes = []
for _n in EXPORTS[:-3]:
    getattr(_lib, _n).restype = _i64 if _n.endswith(("_workspace", "_padded_rows")) else _i32


def library() -> ctypes.CDLL:
    return _lib


# ------------------------------------------------------------------ C names

def fp8q_quantize_act(x, x_dtype, rows, cols, ldx, tile, q, ldq, s, lds, stream=None) -> int:
    return _lib.fp8q_quantize_act(x, x_dtype, rows, cols, ldx, tile, q, ldq, s, lds, stream)


def fp8q_quantize_weight(w, w_dtype, N, K, ldw, q, ldq, s, lds, stream=None) -> int:
    return _lib.fp8q_quantize_weight(w, w_dtype, N, K, ldw, q, ldq, s, lds, stream)


def fp8q_requant_transpose(q, rows, cols, ldq, s, lds, qt, ldqt, st, ldst, stream=None) -> int:
    return _lib.fp8q_requant_transpose(q, rows, cols, ldq, s, lds, qt, ldqt, st, ldst, stream)


def fp8q_gemm(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc, accumulate,
              stream=None) -> int:
    return _lib.fp8q_gemm(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc,
                          accumulate, stream)


def fp8q_grouped_gemm(a, lda, sa, ldsa, b, ldb, b_group_stride, sb, ldsb, sb_group_stride,
                      group_offsets, G, M_total, N, K, c, c_dtype, ldc, stream=None) -> int:
    return _lib.fp8q_grouped_gemm(a, lda, sa, ldsa, b, ldb, b_group_stride, sb, ldsb,
                                  sb_group_stride, group_offsets, G, M_total, N, K, c, c_dtype, ldc,
                                  stream)


def fp8q_quantize_act_ex(x, x_dtype, rows, cols, ldx, tile, q, ldq, s, lds, scale_mode,
                         stream=None) -> int:
    return _lib.fp8q_quantize_act_ex(x, x_dtype, rows, cols, ldx, tile, q, ldq, s, lds, scale_mode,
                                     stream)


def fp8q_quantize_weight_ex(w, w_dtype, N, K, ldw, q, ldq, s, lds, scale_mode, stream=None) -> int:
    return _lib.fp8q_quantize_weight_ex(w, w_dtype, N, K, ldw, q, ldq, s, lds, scale_mode, stream)


def fp8q_requant_transpose_ex(q, rows, cols, ldq, s, lds, qt, ldqt, st, ldst, scale_mode,
                              stream=None) -> int:
    return _lib.fp8q_requant_transpose_ex(q, rows, cols, ldq, s, lds, qt, ldqt, st, ldst, scale_mode,
                                          stream)


def fp8q_transpose_weight(q, N, K, ldq, s, lds, qt, ldqt, st, ldst, stream=None) -> int:
    return _lib.fp8q_transpose_weight(q, N, K, ldq, s, lds, qt, ldqt, st, ldst, stream)


def fp8q_gather_quantize_act(x, x_dtype, rows_in, cols, ldx, row_index, rows_out, q, ldq, s, lds,
                             scale_mode, stream=None) -> int:
    return _lib.fp8q_gather_quantize_act(x, x_dtype, rows_in, cols, ldx, row_index, rows_out, q, ldq, s,
                                         lds, scale_mode, stream)


def fp8q_gemm_ex(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc, accumulate,
                 flags, stream=None) -> int:
    return _lib.fp8q_gemm_ex(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc,
                             accumulate, flags, stream)


def fp8q_grouped_gemm_ex(a, lda, sa, ldsa, b, ldb, b_group_stride, sb, ldsb, sb_group_stride,
                         group_offsets, G, M_total, N, K, c, c_dtype, ldc, flags, stream=None) -> int:
    return _lib.fp8q_grouped_gemm_ex(a, lda, sa, ldsa, b, ldb, b_group_stride, sb, ldsb,
                                     sb_group_stride, group_offsets, G, M_total, N, K, c, c_dtype,
                                     ldc, flags, stream)


def fp8q_gemm_splitk(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc, accumulate,
                     flags, workspace, workspace_bytes, stream=None) -> int:
    return _lib.fp8q_gemm_splitk(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc,
                                 accumulate, flags, workspace, workspace_bytes, stream)


def fp8q_gemm_splitk_noalloc(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc, accumulate,
                             flags, stream=None) -> int:
    return _lib.fp8q_gemm_splitk_noalloc(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc,
                                         accumulate, flags, stream)


SPLITK_SCRATCH_BYTES = 64 << 20


def fp8q_clock_probe(out, ticks, stream=None) -> int:
    return _lib.fp8q_clock_probe(out, ticks, stream)


def fp8q_gemm_splitk_workspace(M, N, K) -> int:
    return _lib.fp8q_gemm_splitk_workspace(M, N, K)


def fp8q_layernorm(x, x_dtype, rows, cols, ldx, gamma, beta, w_dtype, eps, kind, y, y_dtype, ldy, q, ldq, s, lds,
                   scale_mode, mean, rstd, stream=None) -> int:
    return _lib.fp8q_layernorm(x, x_dtype, rows, cols, ldx, gamma, beta, w_dtype, eps, kind, y, y_dtype, ldy, q, ldq,
                               s, lds, scale_mode, mean, rstd, stream)


def fp8q_layernorm_backward_workspace(rows, cols) -> int:
    return _lib.fp8q_layernorm_backward_workspace(rows, cols)


def fp8q_layernorm_backward(dy, lddy, x, ldx, dtype, rows, cols, gamma, w_dtype, mean, rstd, kind, skip, ldskip, dx,
                            lddx, dgamma, dbeta, accumulate, workspace, workspace_bytes, stream=None) -> int:
    return _lib.fp8q_layernorm_backward(dy, lddy, x, ldx, dtype, rows, cols, gamma, w_dtype, mean, rstd, kind, skip,
                                        ldskip, dx, lddx, dgamma, dbeta, accumulate, workspace, workspace_bytes,
                                        stream)


def fp8q_swiglu_quantize(g, u, dtype, ldgu, rows, cols, qh, ldqh, sh, ldsh, qg, qu, ldq, sg, su, lds, scale_mode,
                         stream=None) -> int:
    return _lib.fp8q_swiglu_quantize(g, u, dtype, ldgu, rows, cols, qh, ldqh, sh, ldsh, qg, qu, ldq, sg, su, lds,
                                     scale_mode, stream)


def fp8q_swiglu_backward(qg, qu, ldq, sg, su, lds, dh, dtype, lddh, rows, cols, dg, du, ldd, stream=None) -> int:
    return _lib.fp8q_swiglu_backward(qg, qu, ldq, sg, su, lds, dh, dtype, lddh, rows, cols, dg, du, ldd, stream)


def fp8q_swiglu_backward_quantize(qg, qu, ldq, sg, su, lds, dh, dtype, lddh, rows, cols, qdg, qdu, ldqd, sdg, sdu,
                                  ldsd, qdgt, qdut, ldqt, sdgt, sdut, ldst, qht, ldqht, sht, ldsht, scale_mode,
                                  stream=None) -> int:
    return _lib.fp8q_swiglu_backward_quantize(qg, qu, ldq, sg, su, lds, dh, dtype, lddh, rows, cols, qdg, qdu, ldqd,
                                              sdg, sdu, ldsd, qdgt, qdut, ldqt, sdgt, sdut, ldst, qht, ldqht, sht,
                                              ldsht, scale_mode, stream)


def fp8q_moe_decode_workspace(tokens, hidden, inner, experts, top_k) -> int:
    return _lib.fp8q_moe_decode_workspace(tokens, hidden, inner, experts, top_k)


def fp8q_moe_decode(x, ldx, tokens, hidden, logits, ldl, experts, top_k, renormalize, inner, w_gu, ldw_gu,
                    w_gu_stride, s_gu, lds_gu, s_gu_stride, w_down, ldw_down, w_down_stride, s_down, lds_down,
                    s_down_stride, y, y_dtype, ldy, workspace, workspace_bytes, stream=None) -> int:
    return _lib.fp8q_moe_decode(x, ldx, tokens, hidden, logits, ldl, experts, top_k, renormalize, inner, w_gu, ldw_gu,
                                w_gu_stride, s_gu, lds_gu, s_gu_stride, w_down, ldw_down, w_down_stride, s_down,
                                lds_down, s_down_stride, y, y_dtype, ldy, workspace, workspace_bytes, stream)


def fp8q_grouped_padded_rows(rows, G) -> int:
    return _lib.fp8q_grouped_padded_rows(rows, G)


def fp8q_grouped_quantize_act(x, x_dtype, rows, cols, ldx, group_offsets, G, qt, ldqt, st, ldst, scale_mode,
                              stream=None) -> int:
    return _lib.fp8q_grouped_quantize_act(x, x_dtype, rows, cols, ldx, group_offsets, G, qt, ldqt, st, ldst,
                                          scale_mode, stream)


def fp8q_grouped_requant_transpose(q, rows, cols, ldq, s, lds, group_offsets, G, qt, ldqt, st, ldst, scale_mode,
                                   stream=None) -> int:
    return _lib.fp8q_grouped_requant_transpose(q, rows, cols, ldq, s, lds, group_offsets, G, qt, ldqt, st, ldst,
                                               scale_mode, stream)


def fp8q_grouped_wgrad_workspace(rows, G, N, K) -> int:
    return _lib.fp8q_grouped_wgrad_workspace(rows, G, N, K)


def fp8q_grouped_wgrad(a, lda, sa, ldsa, b, ldb, sb, ldsb, group_offsets, G, rows, N, K, dw, dw_dtype, lddw,
                       dw_group_stride, accumulate, flags, workspace, workspace_bytes, stream=None) -> int:
    return _lib.fp8q_grouped_wgrad(a, lda, sa, ldsa, b, ldb, sb, ldsb, group_offsets, G, rows, N, K, dw, dw_dtype,
                                   lddw, dw_group_stride, accumulate, flags, workspace, workspace_bytes, stream)


def fp8q_adamw(tensors, count, g_dtype, bits, config, scale_mode, stream=None) -> int:
    """tensors: an array of fp8q_adamw_tensor (or its address); config: a fp8q_adamw_config."""
    return _lib.fp8q_adamw(tensors, count, g_dtype, bits, None if config is None else ctypes.addressof(config),
                           scale_mode, stream)


NORM_MAX_COLS = 16384
MOE_MAX_TOKENS = 64
MOE_MAX_TOP_K = 32


def fp8q_strerror(status: int) -> str:
    return _lib.fp8q_strerror(status).decode()


def fp8q_version() -> int:
    return _lib.fp8q_version()


# ------------------------------------------------------------------ helpers

class Fp8qError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {fp8q_strerror(status)} (status {status})")
        self.status = status


def _check(status: int, what: str) -> None:
    if status != FP8Q_OK:
        raise Fp8qError(status, what)


# Not a documented function of torch; the documented one makes a Stream object, 3 us a call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream() -> int:
    """Handle of torch's current stream."""
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return FP8Q_F32
    if t.dtype == torch.bfloat16:
        return FP8Q_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ld(t: torch.Tensor) -> int:
    """Row stride in elements.  A single-row tensor may carry any stride (its
    row stride never multiplies a nonzero index), so report the smallest value
    that satisfies the library's 16-byte rule for that dtype."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (shape[1] > 1 and stride[1] != 1):
        raise ValueError("expected a 2-D tensor with unit column stride")
    if shape[0] <= 1:
        per16 = max(1, 16 // t.element_size())
        return max(per16, -(-shape[1] // per16) * per16)
    return stride[0]


def _on_device(what: str, *ts: torch.Tensor) -> None:
    """Every tensor on the same HIP device (a host tensor's data_ptr would be
    handed to a kernel)."""
    dev = None
    for t in ts:
        if not t.is_cuda:
            raise ValueError(f"{what}: tensors must be on a HIP device")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{what}: tensors on different devices ({dev}, {t.device})")


def _check_codes(what: str, t: torch.Tensor) -> None:
    if t.element_size() != 1 or t.is_floating_point():
        raise ValueError(f"{what}: codes must be a 1-byte integer tensor (uint8 E4M3 bytes), got {t.dtype}")


def _check_scales(what: str, t: torch.Tensor, rows: int, cols: int) -> None:
    """float32 scales, 2-D, at least rows x cols with unit column stride."""
    if t.dtype != torch.float32:
        raise ValueError(f"{what}: scales must be float32, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] < rows or t.shape[1] < cols or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: scales of shape {tuple(t.shape)} do not hold [{rows}][{cols}]")


def _pad16(n: int) -> int:
    return (n + 15) // 16 * 16


def _codes(rows: int, cols: int, device) -> torch.Tensor:
    """uint8 [rows][cols] with a 16-byte-multiple row stride."""
    ld = _pad16(max(cols, 1))
    buf = torch.empty((rows, ld), dtype=torch.uint8, device=device)
    return buf if ld == cols else buf.as_strided((rows, cols), (ld, 1))


def _cdiv(a: int, b: int) -> int:
    return -(-a // b)


def quantize_act(x: torch.Tensor, tile: int = FP8Q_TILE_1x128,
                 scale_mode: int = FP8Q_SCALE_FP32) -> Tuple[torch.Tensor, torch.Tensor]:
    """1x128: returns codes [rows][cols] and scales [ceil(cols/128)][rows].
    128x1: returns codes [cols][rows] (transposed) and scales [ceil(rows/128)][cols]."""
    _on_device("quantize_act", x)
    rows, cols = x.shape
    if tile == FP8Q_TILE_1x128:
        q = _codes(rows, cols, x.device)
        s = torch.empty((_cdiv(cols, 128), rows), dtype=torch.float32, device=x.device)
    else:
        q = _codes(cols, rows, x.device)
        s = torch.empty((_cdiv(rows, 128), cols), dtype=torch.float32, device=x.device)
    args = (x.data_ptr(), _dtype_code(x), rows, cols, _ld(x), tile, q.data_ptr(), _ld(q), s.data_ptr(),
            max(s.stride(0), 1))
    if scale_mode == FP8Q_SCALE_FP32:
        _check(fp8q_quantize_act(*args, _stream()), "fp8q_quantize_act")
    else:
        _check(fp8q_quantize_act_ex(*args, scale_mode, _stream()), "fp8q_quantize_act_ex")
    return q, s


def gather_quantize_act(x: torch.Tensor, row_index: torch.Tensor,
                        scale_mode: int = FP8Q_SCALE_FP32) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows x[row_index[i]] quantized per 1x128 tile (an out-of-range index
    gives a zero row).  row_index: int32 on the device.  Returns codes
    [len][cols] and scales [ceil(cols/128)][len]."""
    if row_index.dtype != torch.int32 or row_index.dim() != 1 or not row_index.is_contiguous():
        raise ValueError("row_index must be a contiguous 1-D int32 tensor")
    _on_device("gather_quantize_act", x, row_index)
    rows_in, cols = x.shape
    rows_out = row_index.numel()
    q = _codes(rows_out, cols, x.device)
    s = torch.empty((_cdiv(cols, 128), rows_out), dtype=torch.float32, device=x.device)
    _check(fp8q_gather_quantize_act(x.data_ptr(), _dtype_code(x), rows_in, cols, _ld(x), row_index.data_ptr(),
                                    rows_out, q.data_ptr(), _ld(q), s.data_ptr(), max(s.stride(0), 1),
                                    scale_mode, _stream()),
           "fp8q_gather_quantize_act")
    return q, s


def quantize_weight(w: torch.Tensor, scale_mode: int = FP8Q_SCALE_FP32) -> Tuple[torch.Tensor, torch.Tensor]:
    """Returns codes [N][K] and 128x128 block scales [ceil(N/128)][ceil(K/128)]."""
    _on_device("quantize_weight", w)
    N, K = w.shape
    q = _codes(N, K, w.device)
    s = torch.empty((_cdiv(N, 128), _cdiv(K, 128)), dtype=torch.float32, device=w.device)
    args = (w.data_ptr(), _dtype_code(w), N, K, _ld(w), q.data_ptr(), _ld(q), s.data_ptr(),
            max(s.stride(0), 1))
    if scale_mode == FP8Q_SCALE_FP32:
        _check(fp8q_quantize_weight(*args, _stream()), "fp8q_quantize_weight")
    else:
        _check(fp8q_quantize_weight_ex(*args, scale_mode, _stream()), "fp8q_quantize_weight_ex")
    return q, s


def requant_transpose(q: torch.Tensor, s: torch.Tensor,
                      scale_mode: int = FP8Q_SCALE_FP32) -> Tuple[torch.Tensor, torch.Tensor]:
    """Cached 1x128 codes q[rows][cols] + scales s[ceil(cols/128)][rows] ->
    128x1 codes qt[cols][rows] + scales st[ceil(rows/128)][cols]."""
    _check_codes("requant_transpose codes", q)
    rows, cols = q.shape
    _check_scales("requant_transpose scales (layout [ceil(cols/128)][rows])", s, _cdiv(cols, 128), rows)
    _on_device("requant_transpose", q, s)
    qt = _codes(cols, rows, q.device)
    st = torch.empty((_cdiv(rows, 128), cols), dtype=torch.float32, device=q.device)
    args = (q.data_ptr(), rows, cols, _ld(q), s.data_ptr(), _ld(s), qt.data_ptr(), _ld(qt), st.data_ptr(),
            max(st.stride(0), 1))
    if scale_mode == FP8Q_SCALE_FP32:
        _check(fp8q_requant_transpose(*args, _stream()), "fp8q_requant_transpose")
    else:
        _check(fp8q_requant_transpose_ex(*args, scale_mode, _stream()), "fp8q_requant_transpose_ex")
    return qt, st


def transpose_weight(q: torch.Tensor, s: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Cached weight codes q[N][K] + block scales s[ceil(N/128)][ceil(K/128)] ->
    qt[K][N] + st[ceil(K/128)][ceil(N/128)] (the Dgrad operand, exact)."""
    _check_codes("transpose_weight codes", q)
    N, K = q.shape
    _check_scales("transpose_weight scales (layout [ceil(N/128)][ceil(K/128)])", s, _cdiv(N, 128), _cdiv(K, 128))
    _on_device("transpose_weight", q, s)
    qt = _codes(K, N, q.device)
    st = torch.empty((_cdiv(K, 128), _cdiv(N, 128)), dtype=torch.float32, device=q.device)
    _check(fp8q_transpose_weight(q.data_ptr(), N, K, _ld(q), s.data_ptr(), _ld(s), qt.data_ptr(), _ld(qt),
                                 st.data_ptr(), _ld(st), _stream()),
           "fp8q_transpose_weight")
    return qt, st


def dgrad(dy_q: torch.Tensor, dy_s: torch.Tensor, wt_q: torch.Tensor, wt_s: torch.Tensor,
          out_dtype: torch.dtype = torch.bfloat16, flags: int = 0) -> torch.Tensor:
    """dX[M][K] = dY[M][N] W[N][K] from dY's 1x128 codes/scales and the
    transposed weight of transpose_weight()."""
    return gemm(dy_q, dy_s, wt_q, wt_s, bscale=FP8Q_BSCALE_BLOCK128, out_dtype=out_dtype, flags=flags)


def gemm(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
         bscale: int = FP8Q_BSCALE_BLOCK128, out_dtype: torch.dtype = torch.bfloat16,
         c: Optional[torch.Tensor] = None, accumulate: bool = False, flags: int = 0,
         split_k: bool = True) -> torch.Tensor:
    """C[M][N] = block-scaled A[M][K] . B[N][K]^T (see fp8q_gemm; `flags`
    selects the matrix-core datapath, see fp8q_gemm_ex).  With split_k, shapes
    that leave the GPU mostly idle run through fp8q_gemm_splitk with a
    workspace allocated here."""
    M, K = a.shape
    N = b.shape[0]
    if b.dim() != 2 or b.shape[1] != K:
        raise ValueError(f"gemm: A is [{M}][{K}] but B is {tuple(b.shape)}; B must be [N][{K}]")
    _check_codes("gemm A", a)
    _check_codes("gemm B", b)
    _check_scales("gemm s_a (layout [K/128][M])", sa, K // 128, M)
    if bscale == FP8Q_BSCALE_BLOCK128:
        _check_scales("gemm s_b (BLOCK128 layout [ceil(N/128)][K/128])", sb, _cdiv(N, 128), K // 128)
    else:
        _check_scales("gemm s_b (ROW layout [K/128][N])", sb, K // 128, N)
    _on_device("gemm", a, sa, b, sb, *(() if c is None else (c,)))
    if c is None:
        c = torch.empty((M, N), dtype=out_dtype, device=a.device)
    elif c.dim() != 2 or tuple(c.shape) != (M, N):
        raise ValueError(f"gemm: C is {tuple(c.shape)}, expected [{M}][{N}]")
    args = (a.data_ptr(), _ld(a), sa.data_ptr(), _ld(sa), b.data_ptr(), _ld(b), sb.data_ptr(), _ld(sb),
            bscale, M, N, K, c.data_ptr(), _dtype_code(c), _ld(c), 1 if accumulate else 0)
    need = fp8q_gemm_splitk_workspace(M, N, K) if split_k else 0
    if need > 0:
        ws = torch.empty(need + 256, dtype=torch.uint8, device=a.device)
        base = (ws.data_ptr() + 255) // 256 * 256
        _check(fp8q_gemm_splitk(*args, flags, base, need, _stream()), "fp8q_gemm_splitk")
    elif flags:
        _check(fp8q_gemm_ex(*args, flags, _stream()), "fp8q_gemm_ex")
    else:
        _check(fp8q_gemm(*args, _stream()), "fp8q_gemm")
    return c


def grouped_gemm(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
                 offsets: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                 c: Optional[torch.Tensor] = None, flags: int = 0) -> torch.Tensor:
    """Per-expert block-scaled GEMM.  a [M_total][K] grouped by expert,
    b [G][N][K] codes, sb [G][ceil(N/128)][K/128], offsets int32 [G+1] on device."""
    M, K = a.shape
    G, N, Kb = b.shape
    if Kb != K or offsets.dtype != torch.int32 or offsets.numel() != G + 1:
        raise ValueError("grouped_gemm: shape mismatch")
    if b.stride(2) != 1 or sb.stride(2) != 1:
        raise ValueError("grouped_gemm: unit inner stride required")
    _check_codes("grouped_gemm A", a)
    _check_codes("grouped_gemm B", b)
    _check_scales("grouped_gemm s_a (layout [K/128][M_total])", sa, K // 128, M)
    if sb.dtype != torch.float32 or sb.dim() != 3 or sb.shape[0] != G or sb.shape[1] < _cdiv(N, 128) \
            or sb.shape[2] < K // 128:
        raise ValueError(f"grouped_gemm: s_b {tuple(sb.shape)} {sb.dtype}, expected float32 "
                         f"[{G}][{_cdiv(N, 128)}][{K // 128}]")
    _on_device("grouped_gemm", a, sa, b, sb, offsets, *(() if c is None else (c,)))
    if c is None:
        c = torch.empty((M, N), dtype=out_dtype, device=a.device)
    args = (a.data_ptr(), _ld(a), sa.data_ptr(), _ld(sa), b.data_ptr(), b.stride(1), b.stride(0),
            sb.data_ptr(), sb.stride(1), sb.stride(0), offsets.data_ptr(), G, M, N, K, c.data_ptr(),
            _dtype_code(c), _ld(c))
    if flags:
        _check(fp8q_grouped_gemm_ex(*args, flags, _stream()), "fp8q_grouped_gemm_ex")
    else:
        _check(fp8q_grouped_gemm(*args, _stream()), "fp8q_grouped_gemm")
    return c


# ------------------------------------------------------------------ feed-forward block
# Calls of few rows take as long as their host code: the library's functions
# are called without the wrappers above.

def _rows(rows: int, cols: int, dtype: torch.dtype, device) -> torch.Tensor:
    """[rows][cols] whose row stride is a multiple of 16 bytes."""
    per16 = 16 // dtype.itemsize
    ld = _cdiv(max(cols, 1), per16) * per16
    buf = torch.empty((rows, ld), dtype=dtype, device=device)
    return buf if ld == cols else buf.as_strided((rows, cols), (ld, 1))


def _scales(groups: int, n: int, device) -> torch.Tensor:
    return torch.empty((groups, n), dtype=torch.float32, device=device)


def _workspace(need: int, device) -> Tuple[Optional[torch.Tensor], int]:
    """A buffer that holds `need` bytes at a 256-byte aligned address, and that address."""
    if need == 0:
        return None, 0
    ws = torch.empty(need + 256, dtype=torch.uint8, device=device)
    return ws, (ws.data_ptr() + 255) // 256 * 256


def _like(what: str, name: str, t: torch.Tensor, ref: torch.Tensor) -> None:
    if t.shape != ref.shape or t.dtype != ref.dtype:
        raise ValueError(f"{what}: {name} is {tuple(t.shape)} {t.dtype}, expected {tuple(ref.shape)} {ref.dtype}")


def _check_vector(what: str, name: str, t: torch.Tensor, n: int, dtype: Optional[torch.dtype] = None) -> None:
    if t.dim() != 1 or t.numel() != n or (n > 1 and t.stride(0) != 1) or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{what}: {name} must be a contiguous vector of {n}"
                         f"{'' if dtype is None else f' {dtype}'}, got {tuple(t.shape)} {t.dtype}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


class LayernormOut(NamedTuple):
    """What layernorm() gives: 1x128 codes and scales, the values, and the rows' statistics; None where not asked
    for (mean: layer norm only)."""
    q: Optional[torch.Tensor]
    s: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    mean: Optional[torch.Tensor]
    rstd: torch.Tensor


def layernorm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
              eps: float = 1e-5, kind: int = FP8Q_NORM_LAYER, quantize: bool = True,
              out_dtype: Optional[torch.dtype] = None, scale_mode: int = FP8Q_SCALE_FP32) -> LayernormOut:
    """Layer norm (FP8Q_NORM_RMS: RMS norm) of the rows of x, into the next GEMM's FP8 operand (`quantize`) and/or
    values of `out_dtype`; see fp8q_layernorm."""
    rows, cols = x.shape
    if not quantize and out_dtype is None:
        raise ValueError("layernorm: nothing to compute (quantize=False and no out_dtype)")
    given = [w for w in (gamma, beta) if w is not None]
    for name, w in (("gamma", gamma), ("beta", beta)):
        if w is not None:
            _check_vector("layernorm", name, w, cols, given[0].dtype)
    _on_device("layernorm", x, *given)
    dev = x.device
    groups = _cdiv(cols, 128) if quantize else 0
    q = _codes(rows, cols, dev) if quantize else None
    y = _rows(rows, cols, out_dtype, dev) if out_dtype is not None else None
    small = torch.empty((groups + 2) * rows, dtype=torch.float32, device=dev)  # scales, rstd, mean
    if cols == 0:  # nothing is launched: the statistics of nothing
        small.fill_(float("nan"))
    s = small.as_strided((groups, rows), (rows, 1)) if quantize else None
    rstd = small.as_strided((rows,), (1,), groups * rows)
    mean = small.as_strided((rows,), (1,), (groups + 1) * rows) if kind == FP8Q_NORM_LAYER else None
    _check(_lib.fp8q_layernorm(x.data_ptr(), _dtype_code(x), rows, cols, _ld(x), _ptr(gamma), _ptr(beta),
                               _dtype_code(given[0]) if given else FP8Q_F32, eps, kind, _ptr(y),
                               FP8Q_F32 if y is None else _dtype_code(y), 0 if y is None else _ld(y), _ptr(q),
                               0 if q is None else _pad16(max(cols, 1)), _ptr(s), max(rows, 1), scale_mode, _ptr(mean),
                               rstd.data_ptr(), _stream()), "fp8q_layernorm")
    return LayernormOut(q, s, y, mean, rstd)


def layernorm_backward(dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor],
                       mean: Optional[torch.Tensor], rstd: torch.Tensor, skip: Optional[torch.Tensor] = None,
                       kind: int = FP8Q_NORM_LAYER, dgamma: Optional[torch.Tensor] = None,
                       dbeta: Optional[torch.Tensor] = None, accumulate: bool = False
                       ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(dx, dgamma, dbeta) of layernorm(); dbeta only for a layer norm or where given.  `skip` is added to dx;
    with `accumulate` the sums are added to the given fp32 dgamma / dbeta.  See fp8q_layernorm_backward."""
    rows, cols = x.shape
    _like("layernorm_backward", "dy", dy, x)
    if skip is not None:
        _like("layernorm_backward", "skip", skip, x)
    if accumulate and dgamma is None:
        raise ValueError("layernorm_backward: accumulate needs the gradients to add to")
    if gamma is not None:
        _check_vector("layernorm_backward", "gamma", gamma, cols)
    if kind == FP8Q_NORM_LAYER:
        if mean is None or (accumulate and dbeta is None):
            raise ValueError("layernorm_backward: a layer norm needs mean (and dbeta to accumulate into)")
        _check_vector("layernorm_backward", "mean", mean, rows, torch.float32)
    _check_vector("layernorm_backward", "rstd", rstd, rows, torch.float32)
    dev = x.device
    if dgamma is None:
        dgamma = torch.empty(cols, dtype=torch.float32, device=dev)
    if dbeta is None and kind == FP8Q_NORM_LAYER:
        dbeta = torch.empty(cols, dtype=torch.float32, device=dev)
    for name, w in (("dgamma", dgamma), ("dbeta", dbeta)):
        if w is not None:
            _check_vector("layernorm_backward", name, w, cols, torch.float32)
    _on_device("layernorm_backward", dy, x, rstd,
               *(t for t in (gamma, mean, skip, dgamma, dbeta) if t is not None))
    dx = _rows(rows, cols, x.dtype, dev)
    need = _lib.fp8q_layernorm_backward_workspace(rows, cols)
    ws, base = _workspace(need, dev)
    _check(_lib.fp8q_layernorm_backward(dy.data_ptr(), _ld(dy), x.data_ptr(), _ld(x), _dtype_code(x), rows, cols,
                                        _ptr(gamma), FP8Q_F32 if gamma is None else _dtype_code(gamma),
                                        _ptr(mean) if kind == FP8Q_NORM_LAYER else None, rstd.data_ptr(), kind,
                                        _ptr(skip), 0 if skip is None else _ld(skip), dx.data_ptr(), _ld(dx),
                                        dgamma.data_ptr(), _ptr(dbeta), 1 if accumulate else 0, base, need, _stream()),
           "fp8q_layernorm_backward")
    return dx, dgamma, dbeta


class SwigluCheckpoint(NamedTuple):
    """The SwiGLU's inputs in 8 bits: 1x128 codes [rows][cols] of gate and up, scales [ceil(cols/128)][rows]."""
    qg: torch.Tensor
    qu: torch.Tensor
    sg: torch.Tensor
    su: torch.Tensor


def _pair(rows: int, cols: int, dtype: torch.dtype, device) -> Tuple[torch.Tensor, torch.Tensor]:
    """Two [rows][cols] halves side by side in one buffer, each row of a half on 16 bytes."""
    per16 = 16 // dtype.itemsize
    ld = _cdiv(max(cols, 1), per16) * per16
    both = torch.empty((rows, 2 * ld), dtype=dtype, device=device)
    return both.as_strided((rows, cols), (2 * ld, 1)), both.as_strided((rows, cols), (2 * ld, 1), ld)


def _stack(groups: int, n: int, dtype: torch.dtype, device) -> Tuple[torch.Tensor, torch.Tensor]:
    """Two [groups][n] halves, one below the other, row stride a multiple of 16 bytes for codes."""
    ld = n if dtype == torch.float32 else _pad16(max(n, 1))
    both = torch.empty((2 * groups, ld), dtype=dtype, device=device)
    return both.as_strided((groups, n), (ld, 1)), both.as_strided((groups, n), (ld, 1), groups * ld)


def swiglu_quantize(g: torch.Tensor, u: torch.Tensor, checkpoint: bool = True, scale_mode: int = FP8Q_SCALE_FP32
                    ) -> Tuple[torch.Tensor, torch.Tensor, Optional[SwigluCheckpoint]]:
    """SwiGLU of gate g and up u [rows][cols] into the down projection's operand: (codes, scales, checkpoint of g
    and u or None).  g and u are the halves of a fused product, or two tensors with the same row stride."""
    _like("swiglu_quantize", "u", u, g)
    rows, cols = g.shape
    ldgu = _ld(g)
    if ldgu != _ld(u):
        raise ValueError(f"swiglu_quantize: row strides {ldgu} and {_ld(u)} differ")
    _on_device("swiglu_quantize", g, u)
    dev, groups = g.device, _cdiv(cols, 128)
    qh, sh = _codes(rows, cols, dev), _scales(groups, rows, dev)
    kept = None
    if checkpoint:
        kept = SwigluCheckpoint(*_pair(rows, cols, torch.uint8, dev), *_stack(groups, rows, torch.float32, dev))
    _check(_lib.fp8q_swiglu_quantize(g.data_ptr(), u.data_ptr(), _dtype_code(g), ldgu, rows, cols, qh.data_ptr(),
                                     _pad16(max(cols, 1)), sh.data_ptr(), max(rows, 1),
                                     *((None, None, 0, None, None, 0) if kept is None else
                                       (kept.qg.data_ptr(), kept.qu.data_ptr(), _ld(kept.qg), kept.sg.data_ptr(),
                                        kept.su.data_ptr(), max(rows, 1))),
                                     scale_mode, _stream()), "fp8q_swiglu_quantize")
    return qh, sh, kept


def _check_checkpoint(what: str, kept: SwigluCheckpoint, dh: torch.Tensor) -> None:
    rows, cols = shape = dh.shape
    qg, qu, sg, su = kept
    for t in (qg, qu):
        _check_codes(what, t)
        if t.shape != shape:
            raise ValueError(f"{what}: checkpoint {tuple(t.shape)}, gradient {tuple(shape)}")
    for t in (sg, su):
        _check_scales(what, t, _cdiv(cols, 128), rows)
    if _ld(qg) != _ld(qu) or (sg.shape[0] > 1 and sg.stride(0) != su.stride(0)):
        raise ValueError(f"{what}: the strides of the checkpoint's halves differ")
    _on_device(what, qg, qu, sg, su, dh)


def _checkpoint_args(kept: SwigluCheckpoint, dh: torch.Tensor) -> tuple:
    rows, cols = dh.shape
    lds = kept.sg.stride(0) if kept.sg.shape[0] > 1 else rows  # one group may carry any stride
    return (kept.qg.data_ptr(), kept.qu.data_ptr(), _ld(kept.qg), kept.sg.data_ptr(), kept.su.data_ptr(), lds,
            dh.data_ptr(), _dtype_code(dh), _ld(dh), rows, cols)


def swiglu_backward(kept: SwigluCheckpoint, dh: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dg, du) of the SwiGLU at the checkpoint's values, in dh's dtype; halves of one buffer (of [rows][2*cols] where
    cols * dtype is a multiple of 16 bytes)."""
    _check_checkpoint("swiglu_backward", kept, dh)
    rows, cols = dh.shape
    dg, du = _pair(rows, cols, dh.dtype, dh.device)
    _check(_lib.fp8q_swiglu_backward(*_checkpoint_args(kept, dh), dg.data_ptr(), du.data_ptr(), _ld(dg), _stream()),
           "fp8q_swiglu_backward")
    return dg, du


class SwigluGrads(NamedTuple):
    """FP8 operands of the backward GEMMs: gradients of gate and up in 1x128 tiles (q, s: Dgrad) and transposed in
    128x1 tiles (qt, st: Wgrad), and the recomputed h transposed in 128x1 tiles (the down projection's Wgrad)."""
    qdg: torch.Tensor
    qdu: torch.Tensor
    sdg: torch.Tensor
    sdu: torch.Tensor
    qdgt: torch.Tensor
    qdut: torch.Tensor
    sdgt: torch.Tensor
    sdut: torch.Tensor
    qht: torch.Tensor
    sht: torch.Tensor

    def gate_up(self) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
        """The operands of a fused gate|up projection: codes [rows][2*cols] with scales [2*cols/128][rows], and codes
        [2*cols][rows] with scales [ceil(rows/128)][2*cols]; views, for cols a multiple of 128."""
        rows, cols = self.qdg.shape
        if cols % 128 != 0:
            raise ValueError(f"gate_up: {cols} columns are not a multiple of 128")
        groups = self.sdgt.shape[0]
        return (self.qdg.as_strided((rows, 2 * cols), (2 * cols, 1)),
                self.sdg.as_strided((2 * cols // 128, rows), (rows, 1), self.sdg.storage_offset()),
                self.qdgt.as_strided((2 * cols, rows), (self.qdgt.stride(0), 1)),
                self.sdgt.as_strided((groups, 2 * cols), (2 * cols, 1), self.sdgt.storage_offset()))


def swiglu_backward_quantize(kept: SwigluCheckpoint, dh: torch.Tensor, scale_mode: int = FP8Q_SCALE_FP32
                             ) -> SwigluGrads:
    """Every FP8 operand of the block's backward GEMMs from the checkpoint and dh; see
    fp8q_swiglu_backward_quantize."""
    _check_checkpoint("swiglu_backward_quantize", kept, dh)
    rows, cols = dh.shape
    dev, groups, tgroups = dh.device, _cdiv(cols, 128), _cdiv(rows, 128)
    ns, nt = groups * rows, tgroups * cols  # scales of one 1x128 and one 128x1 array
    scales = torch.empty(2 * ns + 3 * nt, dtype=torch.float32, device=dev)
    o = SwigluGrads(*_pair(rows, cols, torch.uint8, dev), scales.as_strided((groups, rows), (rows, 1)),
                    scales.as_strided((groups, rows), (rows, 1), ns), *_stack(cols, rows, torch.uint8, dev),
                    scales.as_strided((tgroups, cols), (2 * cols, 1), 2 * ns),
                    scales.as_strided((tgroups, cols), (2 * cols, 1), 2 * ns + cols), _codes(cols, rows, dev),
                    scales.as_strided((tgroups, cols), (cols, 1), 2 * ns + 2 * nt))
    ldq, ldt = 2 * _pad16(max(cols, 1)), _pad16(max(rows, 1))
    _check(_lib.fp8q_swiglu_backward_quantize(*_checkpoint_args(kept, dh), o.qdg.data_ptr(), o.qdu.data_ptr(), ldq,
                                              o.sdg.data_ptr(), o.sdu.data_ptr(), max(rows, 1), o.qdgt.data_ptr(),
                                              o.qdut.data_ptr(), ldt, o.sdgt.data_ptr(), o.sdut.data_ptr(), 2 * cols,
                                              o.qht.data_ptr(), ldt, o.sht.data_ptr(), max(cols, 1), scale_mode,
                                              _stream()),
           "fp8q_swiglu_backward_quantize")
    return o


def _check_experts(what: str, w: torch.Tensor, s: torch.Tensor, shape: Tuple[int, int, int]) -> None:
    _check_codes(what, w)
    E, N, K = shape
    if tuple(w.shape) != shape or (K > 1 and w.stride(2) != 1):
        raise ValueError(f"{what}: codes {tuple(w.shape)}, expected [{E}][{N}][{K}] with unit inner stride")
    if s.dtype != torch.float32 or tuple(s.shape) != (E, _cdiv(N, 128), _cdiv(K, 128)) or \
            (s.shape[2] > 1 and s.stride(2) != 1):
        raise ValueError(f"{what}: scales {tuple(s.shape)} {s.dtype}, expected float32 "
                         f"[{E}][{_cdiv(N, 128)}][{_cdiv(K, 128)}] with unit inner stride")


def _dense_singles(t: torch.Tensor) -> torch.Tensor:
    """[E][rows][cols] with the strides of a dense array along axes of one element (which may carry any)."""
    se, sr, sc = t.stride()
    sr = sr if t.shape[1] > 1 else t.shape[2]
    return t.as_strided(t.shape, (se if t.shape[0] > 1 else t.shape[1] * sr, sr, sc))


def moe_decode(x: torch.Tensor, logits: torch.Tensor, w_gu: torch.Tensor, s_gu: torch.Tensor, w_down: torch.Tensor,
               s_down: torch.Tensor, top_k: int, renormalize: bool = True,
               out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """A mixture-of-experts layer for up to MOE_MAX_TOKENS tokens: x [tokens][hidden] bf16, router logits
    [tokens][experts] fp32, weights w_gu [experts][2*inner][hidden] (gate rows first) and w_down
    [experts][hidden][inner] as FP8 codes with 128x128 block scales.  See fp8q_moe_decode."""
    if x.dtype != torch.bfloat16 or logits.dtype != torch.float32:
        raise ValueError(f"moe_decode: x must be bfloat16 and logits float32, got {x.dtype} and {logits.dtype}")
    if logits.dim() != 2 or logits.shape[0] != x.shape[0] or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"moe_decode: logits {tuple(logits.shape)} for {x.shape[0]} tokens")
    tokens, hidden = x.shape
    experts = logits.shape[1]
    if w_down.dim() != 3:
        raise ValueError(f"moe_decode: w_down {tuple(w_down.shape)} is not [experts][hidden][inner]")
    inner = w_down.shape[2]
    _check_experts("moe_decode w_gu", w_gu, s_gu, (experts, 2 * inner, hidden))
    _check_experts("moe_decode w_down", w_down, s_down, (experts, hidden, inner))
    _on_device("moe_decode", x, logits, w_gu, s_gu, w_down, s_down)
    if experts == 1 or hidden == 128:
        w_gu, s_gu, w_down, s_down = (_dense_singles(t) for t in (w_gu, s_gu, w_down, s_down))
    y = torch.empty((tokens, hidden), dtype=out_dtype, device=x.device)
    need = _lib.fp8q_moe_decode_workspace(tokens, hidden, inner, experts, top_k)
    ws, base = _workspace(need, x.device)
    _check(_lib.fp8q_moe_decode(x.data_ptr(), _ld(x), tokens, hidden, logits.data_ptr(),
                                experts if tokens <= 1 else logits.stride(0), experts, top_k,
                                1 if renormalize else 0, inner, w_gu.data_ptr(), w_gu.stride(1),
                                w_gu.stride(0), s_gu.data_ptr(), s_gu.stride(1), s_gu.stride(0), w_down.data_ptr(),
                                w_down.stride(1), w_down.stride(0), s_down.data_ptr(), s_down.stride(1),
                                s_down.stride(0), y.data_ptr(), _dtype_code(y), _ld(y), base, need, _stream()),
           "fp8q_moe_decode")
    return y


# ------------------------------------------------------------------ experts' weight gradients, AdamW

def _stream_for(what: str, first: torch.Tensor, *rest: torch.Tensor) -> int:
    """torch's current stream, if every tensor is on the current HIP device (a stream of another device would run
    the call there)."""
    dev = first.get_device()
    for t in rest:
        if t.get_device() != dev:
            raise ValueError(f"{what}: tensors on different devices ({first.device}, {t.device})")
    if dev < 0:
        raise ValueError(f"{what}: tensors must be on a HIP device")
    if dev != torch.cuda.current_device():
        raise ValueError(f"{what}: tensors on {first.device}, the current device is cuda:{torch.cuda.current_device()}")
    return torch.cuda.current_stream().cuda_stream if _raw_stream is None else _raw_stream(dev)


def _groups_of(what: str, offsets: torch.Tensor) -> int:
    """Groups of the offsets: int32 [G+1], dense."""
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.shape[0] < 2 or offsets.stride(0) != 1:
        raise ValueError(f"{what}: offsets must be a contiguous int32 vector of the groups and one more, got "
                         f"{tuple(offsets.shape)} {offsets.dtype}")
    return offsets.shape[0] - 1


class GroupedOperand(NamedTuple):
    """An operand of grouped_wgrad(): codes [channels][padded tokens], every group in whole 128-token chunks, scales
    [chunks][channels], and the rows of all groups together that it was made from."""
    q: torch.Tensor
    s: torch.Tensor
    rows: int


def _grouped_operand(rows: int, cols: int, G: int, device) -> GroupedOperand:
    padded = _lib.fp8q_grouped_padded_rows(rows, G)
    return GroupedOperand(torch.empty((cols, padded), dtype=torch.uint8, device=device),
                          torch.empty((padded // 128, cols), dtype=torch.float32, device=device), rows)


def grouped_quantize_act(x: torch.Tensor, offsets: torch.Tensor, scale_mode: int = FP8Q_SCALE_FP32) -> GroupedOperand:
    """Rows x[offsets[g] .. offsets[g+1]) of each group in 128x1 tiles of their own, transposed; see
    fp8q_grouped_quantize_act.  Codes and scales past the last group's chunks hold what the memory held."""
    G = _groups_of("grouped_quantize_act", offsets)
    rows, cols = x.shape
    stream = _stream_for("grouped_quantize_act", x, offsets)
    o = _grouped_operand(rows, cols, G, x.device)
    _check(_lib.fp8q_grouped_quantize_act(x.data_ptr(), _dtype_code(x), rows, cols, _ld(x), offsets.data_ptr(), G,
                                          o.q.data_ptr(), o.q.shape[1], o.s.data_ptr(), cols, scale_mode, stream),
           "fp8q_grouped_quantize_act")
    return o


def grouped_requant_transpose(q: torch.Tensor, s: torch.Tensor, offsets: torch.Tensor,
                              scale_mode: int = FP8Q_SCALE_FP32) -> GroupedOperand:
    """Cached 1x128 codes q[rows][cols] + scales s[ceil(cols/128)][rows], rows grouped, as grouped_quantize_act()
    gives them; see fp8q_grouped_requant_transpose."""
    _check_codes("grouped_requant_transpose codes", q)
    G = _groups_of("grouped_requant_transpose", offsets)
    rows, cols = q.shape
    _check_scales("grouped_requant_transpose scales (layout [ceil(cols/128)][rows])", s, _cdiv(cols, 128), rows)
    stream = _stream_for("grouped_requant_transpose", q, s, offsets)
    o = _grouped_operand(rows, cols, G, q.device)
    _check(_lib.fp8q_grouped_requant_transpose(q.data_ptr(), rows, cols, _ld(q), s.data_ptr(),
                                               s.stride(0) if s.shape[0] > 1 else max(rows, 1), offsets.data_ptr(), G,
                                               o.q.data_ptr(), o.q.shape[1], o.s.data_ptr(), cols, scale_mode, stream),
           "fp8q_grouped_requant_transpose")
    return o


def grouped_wgrad(dy: GroupedOperand, x: GroupedOperand, offsets: torch.Tensor,
                  out_dtype: torch.dtype = torch.float32, dw: Optional[torch.Tensor] = None, accumulate: bool = False,
                  flags: int = 0) -> torch.Tensor:
    """Weight gradients dW [G][N][K] of all groups from dy (N channels) and x (K channels); with `accumulate` added
    to the given fp32 dw.  See fp8q_grouped_wgrad."""
    G = _groups_of("grouped_wgrad", offsets)
    (qa, sa, rows), (qb, sb, rows_x) = dy, x
    if rows != rows_x:
        raise ValueError(f"grouped_wgrad: operands of {rows} and {rows_x} rows")
    (N, held), (K, held_x) = qa.shape, qb.shape
    padded = _lib.fp8q_grouped_padded_rows(rows, G)
    if held < padded or held_x < padded:
        raise ValueError(f"grouped_wgrad: operands of {held} and {held_x} tokens, {G} groups of {rows} rows take up to "
                         f"{padded}")
    if qa.dtype != torch.uint8 or qb.dtype != torch.uint8:
        _check_codes("grouped_wgrad dy", qa)
        _check_codes("grouped_wgrad x", qb)
    _check_scales("grouped_wgrad dy (layout [chunks][channels])", sa, padded // 128, N)
    _check_scales("grouped_wgrad x (layout [chunks][channels])", sb, padded // 128, K)
    if dw is None:
        if accumulate:
            raise ValueError("grouped_wgrad: accumulate needs the gradient to add to")
        stream = _stream_for("grouped_wgrad", qa, sa, qb, sb, offsets)
        dw = torch.empty((G, N, K), dtype=out_dtype, device=qa.device)
        lddw, sg = max(K, 1), N * max(K, 1)
    else:
        if dw.shape != (G, N, K) or (K > 1 and dw.stride(2) != 1):
            raise ValueError(f"grouped_wgrad: dw is {tuple(dw.shape)}, expected [{G}][{N}][{K}] with unit inner stride")
        stream = _stream_for("grouped_wgrad", qa, sa, qb, sb, offsets, dw)
        lddw = dw.stride(1) if N > 1 else max(K, 1)  # axes of one element may carry any stride
        sg = dw.stride(0) if G > 1 else N * lddw
    need = _lib.fp8q_grouped_wgrad_workspace(rows, G, N, K)
    ws, base = _workspace(need, qa.device)
    _check(_lib.fp8q_grouped_wgrad(qa.data_ptr(), _ld(qa), sa.data_ptr(),
                                   sa.stride(0) if sa.shape[0] > 1 else max(N, 1), qb.data_ptr(),
                                   _ld(qb), sb.data_ptr(),
                                   sb.stride(0) if sb.shape[0] > 1 else max(K, 1), offsets.data_ptr(), G, rows, N, K,
                                   dw.data_ptr(), _dtype_code(dw), lddw, sg, 1 if accumulate else 0, flags, base, need,
                                   stream),
           "fp8q_grouped_wgrad")
    return dw


class AdamwState(NamedTuple):
    """Moments of one tensor of n elements: m and v fp32 [n], or codes [n] of m and sqrt(v) with scales sm and sv
    [ceil(n/128)]."""
    m: torch.Tensor
    v: torch.Tensor
    sm: Optional[torch.Tensor]
    sv: Optional[torch.Tensor]


def adamw_state(p: torch.Tensor, bits: int = 32) -> AdamwState:
    """The moments of p before its first step."""
    if bits not in (8, 32):
        raise ValueError(f"adamw_state: moments of {bits} bits; there are 8 and 32")
    n = p.numel()
    if bits == 32:
        return AdamwState(*(torch.zeros(n, dtype=torch.float32, device=p.device) for _ in range(2)), None, None)
    return AdamwState(*(torch.zeros(n, dtype=torch.uint8, device=p.device) for _ in range(2)),
                      *(torch.zeros(_cdiv(n, 128), dtype=torch.float32, device=p.device) for _ in range(2)))


class WeightCodes(NamedTuple):
    """FP8 codes of weights [N][K] or [G][N][K] and of their transposes: q and s as quantize_weight() gives them for
    each matrix, qt [..][K][N] (row stride a multiple of 16) and st as transpose_weight() does, or None."""
    q: torch.Tensor
    s: torch.Tensor
    qt: Optional[torch.Tensor]
    st: Optional[torch.Tensor]


def weight_codes(w: torch.Tensor, transposed: bool = True, scale_mode: int = FP8Q_SCALE_FP32) -> WeightCodes:
    """The codes of weights w ([N][K] or [G][N][K], K a multiple of 128) that adamw() keeps up to date."""
    if w.dim() not in (2, 3) or w.shape[-1] % 128 != 0 or not w.is_contiguous():
        raise ValueError(f"weight_codes: weights {tuple(w.shape)}, expected dense [N][K] or [G][N][K] with K a multiple of 128")
    _stream_for("weight_codes", w)
    lead, (N, K), dev = w.shape[:-2], w.shape[-2:], w.device
    nb, kb, n16 = _cdiv(N, 128), K // 128, _pad16(N)
    o = WeightCodes(torch.empty((*lead, N, K), dtype=torch.uint8, device=dev),
                    torch.empty((*lead, nb, kb), dtype=torch.float32, device=dev),
                    torch.empty((*lead, K, n16), dtype=torch.uint8, device=dev)[..., :N] if transposed else None,
                    torch.empty((*lead, kb, nb), dtype=torch.float32, device=dev) if transposed else None)
    for g in range(w.shape[0]) if w.dim() == 3 else [...]:
        _check(fp8q_quantize_weight_ex(w[g].data_ptr(), _dtype_code(w), N, K, max(K, 8), o.q[g].data_ptr(), max(K, 16),
                                       o.s[g].data_ptr(), max(kb, 1), scale_mode, _stream()), "fp8q_quantize_weight_ex")
        if transposed:
            _check(fp8q_transpose_weight(o.q[g].data_ptr(), N, K, max(K, 16), o.s[g].data_ptr(), max(kb, 1),
                                         o.qt[g].data_ptr(), max(n16, 16), o.st[g].data_ptr(), max(nb, 1), _stream()),
                   "fp8q_transpose_weight")
    return o


class AdamwTensors:
    """What adamw() works on: made by adamw_tensors(), kept from step to step.  It holds the tensors and the memory that
    they had then, which adamw() reads and writes, and refuses parameters that have got other memory since."""

    def __init__(self, held: tuple, array, g_dtype: int, bits: int, device: torch.device):
        self.held, self.array, self.g_dtype, self.bits, self.device = held, array, g_dtype, bits, device
        params, grads, states, codes = held
        self.params, self.addresses, self.places = list(params), [p.data_ptr() for p in params], list(range(len(params)))
        self.memory = tuple(t.untyped_storage() for ts in (params, grads, *states, *filter(None, codes)) for t in ts
                            if t is not None)
        # what a backward pass may have kept: parameters that autograd follows, and codes
        self.versioned = [p for p in params if p.requires_grad] + [t for c in codes if c is not None for t in c
                                                                   if t is not None]


def _dense(t: torch.Tensor, shape: tuple, dtype: torch.dtype) -> bool:
    return t.shape == shape and t.dtype == dtype and t.is_contiguous()


def _not_dense(at: str, name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype) -> ValueError:
    return ValueError(f"{at}: {name} is {tuple(t.shape)} {t.dtype} with strides {t.stride()}, expected dense "
                      f"{tuple(shape)} {dtype}")


def adamw_tensors(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], states: Sequence[AdamwState],
                  codes: Optional[Sequence[Optional[WeightCodes]]] = None) -> AdamwTensors:
    """Checks the tensors of an optimizer step once: dense fp32 params, grads of the same shapes (all fp32 or all
    bf16), moments of adamw_state() (all of 32 or all of 8 bits), and for weights the codes of weight_codes() or None.
    adamw() then updates params, moments and codes in place, from what grads hold at that time.  A tensor that gets
    other memory (p.data = ..., a new gradient tensor) needs a new list; none may be resized while the list is used."""
    what = "adamw_tensors"
    codes = [None] * len(params) if codes is None else list(codes)
    if not len(params) == len(grads) == len(states) == len(codes):
        raise ValueError(f"{what}: {len(params)} params, {len(grads)} grads, {len(states)} states, {len(codes)} codes")
    if not params:
        raise ValueError(f"{what}: no tensors")
    bits = 8 if states[0].m.dtype == torch.uint8 else 32
    kind, gtype = torch.uint8 if bits == 8 else torch.float32, grads[0].dtype
    array = (fp8q_adamw_tensor * len(params))()
    spans = []  # (first byte, one past the last, written)
    for i, (p, g, (m, v, sm, sv), c) in enumerate(zip(params, grads, states, codes)):
        at, n, shape = f"{what}: tensor {i}", p.numel(), p.shape
        flat = torch.Size((n,))
        checks = [("the parameter", p, shape, torch.float32), ("m", m, flat, kind), ("v", v, flat, kind)]
        if bits == 8:
            if sm is None or sv is None:
                raise ValueError(f"{at}: 8-bit moments need scales")
            tiles = torch.Size((_cdiv(n, 128),))
            checks += [("sm", sm, tiles, torch.float32), ("sv", sv, tiles, torch.float32)]
        elif sm is not None or sv is not None:
            raise ValueError(f"{at}: fp32 moments have no scales")
        d = array[i]
        d.n, d.p, d.g, d.m, d.v = n, p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr()
        if bits == 8:
            d.sm, d.sv = sm.data_ptr(), sv.data_ptr()
        if c is not None and n:
            if p.dim() not in (2, 3) or shape[-1] % 128 != 0:
                raise ValueError(f"{at}: codes are kept of [N][K] or [G][N][K] with K a multiple of 128, not {tuple(shape)}")
            lead, (N, K) = shape[:-2], shape[-2:]
            nb, kb, n16 = _cdiv(N, 128), K // 128, _pad16(N)
            checks += [("q", c.q, shape, torch.uint8), ("s", c.s, torch.Size((*lead, nb, kb)), torch.float32)]
            if (c.qt is None) != (c.st is None):
                raise ValueError(f"{at}: qt and st go together")
            d.N, d.K, d.q, d.s = N, K, c.q.data_ptr(), c.s.data_ptr()
            if c.qt is not None:
                checks.append(("st", c.st, torch.Size((*lead, kb, nb)), torch.float32))
                strides = c.qt.stride()
                if tuple(c.qt.shape) != (*lead, K, N) or c.qt.dtype != torch.uint8 or \
                        (N > 1 and strides[-1] != 1) or strides[-2] != n16 or \
                        (lead and lead[0] > 1 and strides[0] != K * n16):
                    raise ValueError(f"{at}: qt is {tuple(c.qt.shape)} {c.qt.dtype} with strides {strides}, expected "
                                     f"that of weight_codes()")
                _on_device(at, p, c.qt)
                spans.append((c.qt.data_ptr(), c.qt.data_ptr() + n // N * n16 - n16 + N, True))
                d.qt, d.st = c.qt.data_ptr(), c.st.data_ptr()
        for name, t, want, dtype in checks:
            if not _dense(t, want, dtype):
                raise _not_dense(at, name, t, want, dtype)
        if not _dense(g, shape, gtype):
            raise _not_dense(at, "the gradient", g, shape, gtype)
        _on_device(at, g, *(t for _, t, _, _ in checks))
        for _, t, _, _ in checks:
            spans.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), True))
        spans.append((d.g or 0, (d.g or 0) + n * g.element_size(), False))
    _stream_for(what, *params)
    _no_overlap(what, spans)
    return AdamwTensors((tuple(params), tuple(grads), tuple(states), tuple(codes)), array, _dtype_code(grads[0]), bits,
                        params[0].device)


def _no_overlap(what: str, spans: list) -> None:
    """spans: (first byte, one past the last, written).  No byte that is written belongs to two of them."""
    end = end_w = 0  # ends of what was met so far, and of what is written of it
    for lo, hi, w in sorted(s for s in spans if s[0] < s[1]):
        if lo < end_w or (w and lo < end):
            raise ValueError(f"{what}: tensors overlap (each may be in the list once)")
        end = max(end, hi)
        end_w = max(end_w, hi) if w else end_w


def adamw(tensors: AdamwTensors, step: Union[int, torch.Tensor], lr: Union[float, torch.Tensor], beta1: float = 0.9,
          beta2: float = 0.95, eps: float = 1e-8, weight_decay: float = 0.1,
          grad_scale: Optional[torch.Tensor] = None, seed: int = 0, scale_mode: int = FP8Q_SCALE_FP32) -> None:
    """One AdamW step over all the tensors, in place; step counts from 1.  step (int64), lr and grad_scale (fp32) may
    be tensors of one element on the device, read when the step runs: a captured step is then replayed with other
    values.  grad_scale multiplies the gradients; seed chooses the random numbers that round 8-bit moments.  See
    fp8q_adamw.  To autograd the parameters and codes are changed in place: a backward pass that kept them is refused."""
    _not_moved(tensors.params, tensors.addresses, tensors.places)
    c = fp8q_adamw_config(0.0, beta1, beta2, eps, weight_decay, 0, None, None, None, seed & 0xFFFFFFFF)
    if isinstance(step, torch.Tensor):
        c.step_dev = _device_scalar("step", step, torch.int64, tensors)
    else:
        c.step = step
    if isinstance(lr, torch.Tensor):
        c.lr_dev = _device_scalar("lr", lr, torch.float32, tensors)
    else:
        c.lr = lr
    if grad_scale is not None:
        c.grad_scale = _device_scalar("grad_scale", grad_scale, torch.float32, tensors)
    stream = _stream_for("adamw", tensors.held[0][0])
    _check(_lib.fp8q_adamw(tensors.array, len(tensors.array), tensors.g_dtype, tensors.bits, ctypes.addressof(c),
                           scale_mode, stream), "fp8q_adamw")
    if tensors.versioned:
        increment_version(tensors.versioned)


# Not a documented function of torch: one call for all tensors, 1.8 us for 60 of them, where asking each takes 2.6.
_same_addresses = getattr(torch._C, "_tensors_data_ptrs_at_indices_equal", None)


def _not_moved(params: list, addresses: list, places: list) -> None:
    """The parameters stand where they stood when their list was made."""
    if _same_addresses is not None and _same_addresses(params, addresses, places):
        return
    for i, (p, a) in enumerate(zip(params, addresses)):
        if p.data_ptr() != a:
            raise ValueError(f"adamw: parameter {i} has other memory than when its list was made; make a new list")


def _device_scalar(name: str, t: torch.Tensor, dtype: torch.dtype, tensors: AdamwTensors) -> int:
    """Address of one number on the device of the tensors."""
    if t.numel() != 1 or t.dtype != dtype or t.device != tensors.device:
        raise ValueError(f"adamw: {name} must be one {dtype} on {tensors.device}, got {tuple(t.shape)} {t.dtype} on "
                         f"{t.device}")
    return t.data_ptr()
