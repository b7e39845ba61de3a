"""Python binding of libtemx.so, the MXFP8 Linear hot path for MI355X (gfx950).

Every function named ``te_*`` marshals torch tensors (device memory) and the
current HIP stream into the C entry point of the same name declared in
``include/temx.h``; all computation happens in the library's HIP kernels.
The helpers without the prefix only allocate outputs with torch and call the
``te_*`` functions.  There is no fallback: importing this package fails if
the library has not been built (``python mxfp8_mixed_precision_amd/build.py``).
"""

from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtemx.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with `python mxfp8_mixed_precision_amd/build.py`")
_lib = ctypes.CDLL(_LIB_PATH)

# enum values of include/temx.h
TE_OK, TE_ERR_NULL, TE_ERR_SHAPE, TE_ERR_ALIGN, TE_ERR_DTYPE, TE_ERR_WORKSPACE, TE_ERR_HIP, TE_ERR_VALUE, TE_ERR_ARCH = range(9)
TE_BF16, TE_FP32, TE_E4M3, TE_E5M2, TE_E8M0, TE_FP16 = range(6)
TE_EPI_NONE, TE_EPI_BIAS, TE_EPI_BIAS_GELU_AUX, TE_EPI_DGELU, TE_EPI_ACCUMULATE = range(5)
TE_ROWWISE, TE_COLWISE, TE_BOTH = 1, 2, 3
TE_AMAX_MAX, TE_AMAX_MOST_RECENT = 0, 1
AMAX_ALGOS = {"max": TE_AMAX_MAX, "most_recent": TE_AMAX_MOST_RECENT}
TE_BLOCK_SCALES_E8M0, TE_BLOCK_SCALES_FP32 = 0, 1
TE_NORM_LAYER, TE_NORM_RMS = 0, 1
NORM_KINDS = {"layer": TE_NORM_LAYER, "rms": TE_NORM_RMS}
TE_ACT_SILU, TE_ACT_GELU = 0, 1
ACTIVATIONS = {"silu": TE_ACT_SILU, "gelu": TE_ACT_GELU}
TE_SCORE_SOFTMAX, TE_SCORE_SIGMOID = 0, 1
SCORES = {"softmax": TE_SCORE_SOFTMAX, "sigmoid": TE_SCORE_SIGMOID}
TE_W4_INT4, TE_W4_E2M1 = 0, 1
W4_FORMATS = {"int4": TE_W4_INT4, "e2m1": TE_W4_E2M1}
BLOCK_SCALINGS = {"e8m0": TE_BLOCK_SCALES_E8M0, "fp32": TE_BLOCK_SCALES_FP32}

FORMATS = {"e4m3": TE_E4M3, "e5m2": TE_E5M2}
EPILOGUES = {"none": TE_EPI_NONE, "bias": TE_EPI_BIAS, "bias_gelu_aux": TE_EPI_BIAS_GELU_AUX,
             "dgelu": TE_EPI_DGELU, "accumulate": TE_EPI_ACCUMULATE}
DIRECTIONS = {"row": TE_ROWWISE, "col": TE_COLWISE, "both": TE_BOTH}

_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_SIGS = {
    "te_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "te_amax_workspace_size": (_sz, [_i64]),
    "te_amax_reduce": (ctypes.c_int, [_vp, _i64, _vp, _vp, _sz, _vp]),
    "te_fp8_cast_current_scaling": (ctypes.c_int, [_vp, _i64, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "te_fp8_cast_current_scaling_noalloc": (ctypes.c_int, [_vp, _i64, ctypes.c_int, _vp, _vp, _vp, _vp, _vp]),
    "te_fp8_cast_delayed_scaling": (ctypes.c_int, [_vp, _i64, ctypes.c_int, _vp, _vp, _vp, _vp, ctypes.c_int,
                                                   ctypes.c_int, ctypes.c_int, _vp, _sz, _vp]),
    "te_fp8_gemm": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int, _i64, _i64, _i64,
                                   _vp, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _sz, _vp]),
    "te_mxfp8_quantize": (ctypes.c_int, [_vp, _i64, _i64, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _vp, _vp]),
    "te_mxfp8_quantize_bgrad_workspace_size": (_sz, [_i64, _i64]),
    "te_mxfp8_quantize_bgrad": (ctypes.c_int, [_vp, _i64, _i64, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, ctypes.c_int,
                                               _vp, _sz, _vp]),
    "te_mxfp8_gemm_workspace_size": (_sz, [_i64, _i64, _i64]),
    "te_mxfp8_gemm": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int, _i64, _i64, _i64,
                                     _vp, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _sz, _vp]),
    "te_mxfp8_gemm_mxout": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int, _i64, _i64, _i64,
                                           _vp, _vp, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _sz, _vp]),
    "te_mxfp8_grouped_gemm": (ctypes.c_int, [_i32, _vp, _i64, _vp, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int,
                                             _i64, _i64, _vp, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _sz, _vp]),
    "te_fp8_block_quantize": (ctypes.c_int, [_vp, _i64, _i64, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp]),
    "te_fp8_block_scales_to_mx": (ctypes.c_int, [_vp, _i64, _i64, ctypes.c_int, _vp, _vp]),
    "te_fp8_block_gemm_workspace_size": (_sz, [_i64, _i64, _i64, ctypes.c_int]),
    "te_fp8_block_gemm": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int, ctypes.c_int, _i64, _i64,
                                         _i64, _vp, ctypes.c_int, ctypes.c_int, _vp, _vp, ctypes.c_int, ctypes.c_float,
                                         _vp, _sz, _vp]),
    "te_norm_forward": (ctypes.c_int, [ctypes.c_int, _vp, ctypes.c_int, _i64, _i64, _vp, _vp, _vp, ctypes.c_int,
                                       ctypes.c_float, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp]),
    "te_norm_backward_workspace_size": (_sz, [_i64, _i64]),
    "te_norm_backward": (ctypes.c_int, [ctypes.c_int, _vp, _vp, _vp, ctypes.c_int, _i64, _i64, _vp, ctypes.c_int,
                                        _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "te_mxfp8_gated_gemm_workspace_size": (_sz, [_i64, _i64, _i64]),
    "te_mxfp8_gated_gemm": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int, _i64, _i64, _i64,
                                           ctypes.c_int, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _sz, _vp]),
    "te_mxfp8_dgated_gemm_workspace_size": (_sz, [_i64, _i64, _i64]),
    "te_mxfp8_dgated_gemm": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int, _i64, _i64, _i64,
                                            ctypes.c_int, _vp, _vp, _vp, _sz, _vp]),
    "te_mxfp8_grouped_gated_gemm": (ctypes.c_int, [_i32, _vp, _i64, _vp, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int,
                                                   _i64, _i64, ctypes.c_int, _vp, _vp, _vp, _vp]),
    "te_mxfp8_grouped_dgated_gemm": (ctypes.c_int, [_i32, _vp, _i64, _vp, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int,
                                                    _i64, _i64, ctypes.c_int, _vp, _vp, _vp]),
    "te_moe_route": (ctypes.c_int, [ctypes.c_int, _vp, ctypes.c_int, _i64, _i32, _i32, _vp, ctypes.c_int, ctypes.c_float,
                                    _vp, _vp, _vp]),
    "te_moe_route_backward": (ctypes.c_int, [ctypes.c_int, _vp, ctypes.c_int, _i64, _i32, _i32, ctypes.c_int,
                                             ctypes.c_float, _vp, _vp, _vp, _vp]),
    "te_moe_sort_workspace_size": (_sz, [_i64, _i32]),
    "te_moe_sort": (ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "te_moe_dispatch": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _vp, _i32, _i64, _vp, _vp, _vp, ctypes.c_int, _vp]),
    "te_moe_combine": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _vp, _vp, _i64, _i32, _vp, _vp]),
    "te_moe_combine_backward": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _vp, _vp,
                                               ctypes.c_int, _vp, _vp]),
    "te_w4_gemm": (ctypes.c_int, [_vp, ctypes.c_int, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp, _i32, _i64, _i64, _i64,
                                  _vp, ctypes.c_int, _vp, _vp]),
    "te_w4_gated_gemm": (ctypes.c_int, [_vp, ctypes.c_int, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp, _i32, _i64, _i64,
                                        _i64, ctypes.c_int, _vp, ctypes.c_int, _vp, _vp]),
    "te_w4_grouped_gemm": (ctypes.c_int, [_i32, _vp, _i64, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp,
                                          _i32, _i64, _i64, _vp, ctypes.c_int, _vp, _vp]),
    "te_w4_grouped_gated_gemm": (ctypes.c_int, [_i32, _vp, _i64, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp,
                                                ctypes.c_int, _vp, _i32, _i64, _i64, ctypes.c_int, _vp, ctypes.c_int,
                                                _vp, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)
_FNS = {_name: getattr(_lib, _name) for _name in _SIGS}


class TemxError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {te_status_str(status)}")
        self.status = status


def te_status_str(status: int) -> str:
    return _lib.te_status_str(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != TE_OK:
        raise TemxError(fn, status)


def _ptr(t):
    """Device address of a tensor argument.  Every pointer of the C ABI is a device pointer into a dense
    row-major buffer, so host tensors and non-contiguous views are refused here (the library cannot tell
    them apart from valid arguments)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"expected a GPU tensor, got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor (row-major, no strides)")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _fmt(f) -> int:
    return FORMATS[f] if isinstance(f, str) else int(f)


# Argument checks of the wrappers.  The C ABI sees only addresses and sizes, so
# a tensor of the wrong shape or element type would be read or written past
# its end there; every wrapper checks its tensors against the sizes it passes
# before calling the library.
_BYTE_DTYPES = {torch.uint8, torch.int8} | {getattr(torch, n) for n in
                                           ("float8_e4m3fn", "float8_e5m2", "float8_e8m0fnu") if hasattr(torch, n)}
_BF16_DTYPES = {torch.bfloat16, torch.int16} | ({torch.uint16} if hasattr(torch, "uint16") else set())


def _require(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _check_tensor(t, name: str, shape, dtypes, kind: str, optional: bool = False) -> None:
    """t must have exactly `shape` and a dtype in `dtypes` (None is accepted only when optional)."""
    if t is None:
        _require(optional, f"{name} is required")
        return
    _require(t.dtype in dtypes, f"{name}: expected {kind}, got {t.dtype}")
    _require(tuple(t.shape) == tuple(int(v) for v in shape),
             f"{name}: expected shape {tuple(int(v) for v in shape)}, got {tuple(t.shape)}")


def _codes(t, name, shape, optional=False):
    _check_tensor(t, name, shape, _BYTE_DTYPES, "1-byte codes (uint8)", optional)


def _bf16(t, name, shape, optional=False):
    _check_tensor(t, name, shape, _BF16_DTYPES, "bf16 (or its int16 bits)", optional)


def _f32(t, name, shape, optional=False):
    _check_tensor(t, name, shape, {torch.float32}, "float32", optional)


def _scalar_f32(t, name):
    _require(t is not None and t.dtype == torch.float32 and t.numel() >= 1, f"{name}: expected a float32 scalar")


_OUT_DTYPES = {torch.bfloat16: TE_BF16, torch.float32: TE_FP32, torch.float16: TE_FP16}


def _gemm_out(d, name, M, N, epi, allow_fp16=False):
    """D of the bf16/fp32-output GEMMs: [M, N] bf16 or float32 (float16 too where allowed); "accumulate"
    needs float32."""
    kinds = (torch.bfloat16, torch.float32) + ((torch.float16,) if allow_fp16 else ())
    _require(d is not None and d.dtype in kinds,
             f"{name}: expected {' or '.join(str(k).replace('torch.', '') for k in kinds)}, "
             f"got {None if d is None else d.dtype}")
    _require(epi != TE_EPI_ACCUMULATE or d.dtype == torch.float32, f"{name}: the accumulate epilogue needs float32")
    _require(tuple(d.shape) == (M, N), f"{name}: expected shape {(M, N)}, got {tuple(d.shape)}")
    return _OUT_DTYPES[d.dtype]


def _epi_tensors(bias, bias_shape, aux, M, N):
    """bias (bf16, bias_shape) with the bias epilogues; aux (bf16 [M, N]) with GELU aux and dgelu."""
    _bf16(bias, "bias", bias_shape, optional=True)
    _bf16(aux, "aux", (M, N), optional=True)


def _epilogue(epilogue) -> int:
    return EPILOGUES[epilogue] if isinstance(epilogue, str) else int(epilogue)


def _ws_bytes(workspace) -> int:
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------- entry points

def te_amax_workspace_size(n: int) -> int:
    return int(_lib.te_amax_workspace_size(int(n)))


def te_amax_reduce(x, amax_out, workspace, stream=None) -> None:
    _bf16(x, "x", tuple(x.shape))
    _scalar_f32(amax_out, "amax_out")
    _check("te_amax_reduce", _lib.te_amax_reduce(_ptr(x), x.numel(), _ptr(amax_out), _ptr(workspace),
                                                 workspace.numel() * workspace.element_size(), _stream(stream)))


def te_fp8_cast_current_scaling(x, fmt, q_out, amax_out, scale_out, scale_inv_out, workspace, stream=None) -> None:
    _bf16(x, "x", tuple(x.shape))
    _codes(q_out, "q_out", tuple(x.shape))
    for t, n in ((amax_out, "amax_out"), (scale_out, "scale_out"), (scale_inv_out, "scale_inv_out")):
        _scalar_f32(t, n)
    _check("te_fp8_cast_current_scaling", _lib.te_fp8_cast_current_scaling(
        _ptr(x), x.numel(), _fmt(fmt), _ptr(q_out), _ptr(amax_out), _ptr(scale_out), _ptr(scale_inv_out),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def te_fp8_cast_current_scaling_noalloc(x, fmt, q_out, amax_out, scale_out, scale_inv_out, stream=None) -> None:
    _bf16(x, "x", tuple(x.shape))
    _codes(q_out, "q_out", tuple(x.shape))
    for t, n in ((amax_out, "amax_out"), (scale_out, "scale_out"), (scale_inv_out, "scale_inv_out")):
        _scalar_f32(t, n)
    _check("te_fp8_cast_current_scaling_noalloc", _lib.te_fp8_cast_current_scaling_noalloc(
        _ptr(x), x.numel(), _fmt(fmt), _ptr(q_out), _ptr(amax_out), _ptr(scale_out), _ptr(scale_inv_out),
        _stream(stream)))


def te_fp8_cast_delayed_scaling(x, fmt, q_out, q_scale_inv_out, scale, amax_history, workspace, algo="max",
                                margin=0, stream=None) -> None:
    a = AMAX_ALGOS[algo] if isinstance(algo, str) else int(algo)
    _bf16(x, "x", tuple(x.shape))
    _codes(q_out, "q_out", tuple(x.shape))
    _scalar_f32(q_scale_inv_out, "q_scale_inv_out")
    _scalar_f32(scale, "scale")
    _require(amax_history is not None and amax_history.dtype == torch.float32 and amax_history.dim() == 1,
             "amax_history: expected a 1-D float32 tensor")
    _check("te_fp8_cast_delayed_scaling", _lib.te_fp8_cast_delayed_scaling(
        _ptr(x), x.numel(), _fmt(fmt), _ptr(q_out), _ptr(q_scale_inv_out), _ptr(scale), _ptr(amax_history),
        amax_history.numel(), a, int(margin), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def te_fp8_gemm(a, a_scale_inv, a_fmt, b, b_scale_inv, b_fmt, d, epilogue="none", bias=None, aux=None,
                workspace=None, stream=None) -> None:
    _require(a.dim() == 2 and b.dim() == 2, "a and b must be 2-D")
    M, K = a.shape
    N = b.shape[0]
    _codes(a, "a", (M, K))
    _codes(b, "b", (N, K))
    _scalar_f32(a_scale_inv, "a_scale_inv")
    _scalar_f32(b_scale_inv, "b_scale_inv")
    epi = _epilogue(epilogue)
    d_dtype = _gemm_out(d, "d", M, N, epi)
    _epi_tensors(bias, (N,), aux, M, N)
    ws_bytes = _ws_bytes(workspace)
    _check("te_fp8_gemm", _lib.te_fp8_gemm(
        _ptr(a), _ptr(a_scale_inv), _fmt(a_fmt), _ptr(b), _ptr(b_scale_inv), _fmt(b_fmt), M, N, K,
        _ptr(d), d_dtype, epi, _ptr(bias), _ptr(aux), _ptr(workspace), ws_bytes, _stream(stream)))


def te_mxfp8_quantize(x, fmt, direction, q_row=None, s_row=None, q_col=None, s_col=None, stream=None) -> None:
    d = DIRECTIONS[direction] if isinstance(direction, str) else int(direction)
    _require(x.dim() == 2, "x must be 2-D")
    rows, cols = x.shape
    _bf16(x, "x", (rows, cols))
    _codes(q_row, "q_row", (rows, cols), optional=True)
    _codes(s_row, "s_row", (rows, cols // 32), optional=True)
    _codes(q_col, "q_col", (cols, rows), optional=True)
    _codes(s_col, "s_col", (cols, rows // 32), optional=True)
    _check("te_mxfp8_quantize", _lib.te_mxfp8_quantize(
        _ptr(x), rows, cols, _fmt(fmt), d, _ptr(q_row), _ptr(s_row), _ptr(q_col), _ptr(s_col), _stream(stream)))


def te_mxfp8_quantize_bgrad_workspace_size(rows: int, cols: int) -> int:
    return int(_lib.te_mxfp8_quantize_bgrad_workspace_size(int(rows), int(cols)))


def te_mxfp8_quantize_bgrad(x, fmt, q_row, s_row, q_col, s_col, bgrad, workspace, stream=None) -> None:
    _require(x.dim() == 2, "x must be 2-D")
    rows, cols = x.shape
    _bf16(x, "x", (rows, cols))
    empty = rows == 0  # no codes to write: the outputs may be None
    _codes(q_row, "q_row", (rows, cols), optional=empty)
    _codes(s_row, "s_row", (rows, cols // 32), optional=empty)
    _codes(q_col, "q_col", (cols, rows), optional=empty)
    _codes(s_col, "s_col", (cols, rows // 32), optional=empty)
    _check_tensor(bgrad, "bgrad", (cols,), {torch.float32, torch.bfloat16}, "float32 or bfloat16")
    b_dtype = TE_FP32 if bgrad.dtype == torch.float32 else TE_BF16
    ws_bytes = _ws_bytes(workspace)
    _check("te_mxfp8_quantize_bgrad", _lib.te_mxfp8_quantize_bgrad(
        _ptr(x), rows, cols, _fmt(fmt), _ptr(q_row), _ptr(s_row), _ptr(q_col), _ptr(s_col), _ptr(bgrad), b_dtype,
        _ptr(workspace), ws_bytes, _stream(stream)))


def te_mxfp8_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(_lib.te_mxfp8_gemm_workspace_size(M, N, K))


def _mx_operands(a, a_scale, b, b_scale):
    """Shapes of two MXFP8 operands: a [M, K] + [M, K/32], b [N, K] + [N, K/32] -> (M, N, K)."""
    _require(a.dim() == 2 and b.dim() == 2, "a and b must be 2-D")
    M, K = a.shape
    N = b.shape[0]
    _codes(a, "a", (M, K))
    _codes(a_scale, "a_scale", (M, K // 32))
    _codes(b, "b", (N, K))
    _codes(b_scale, "b_scale", (N, K // 32))
    return M, N, K


def te_mxfp8_gemm(a, a_scale, a_fmt, b, b_scale, b_fmt, d, epilogue="none", bias=None, aux=None,
                  workspace=None, stream=None) -> None:
    M, N, K = _mx_operands(a, a_scale, b, b_scale)
    epi = _epilogue(epilogue)
    d_dtype = _gemm_out(d, "d", M, N, epi)
    _epi_tensors(bias, (N,), aux, M, N)
    ws_bytes = _ws_bytes(workspace)
    _check("te_mxfp8_gemm", _lib.te_mxfp8_gemm(
        _ptr(a), _ptr(a_scale), _fmt(a_fmt), _ptr(b), _ptr(b_scale), _fmt(b_fmt), M, N, K,
        _ptr(d), d_dtype, epi, _ptr(bias), _ptr(aux), _ptr(workspace), ws_bytes, _stream(stream)))


def te_mxfp8_gemm_mxout(a, a_scale, a_fmt, b, b_scale, b_fmt, d, d_scale, d_fmt, epilogue="none", bias=None,
                        aux=None, workspace=None, stream=None) -> None:
    M, N, K = _mx_operands(a, a_scale, b, b_scale)
    epi = _epilogue(epilogue)
    _codes(d, "d", (M, N))
    _codes(d_scale, "d_scale", (M, N // 32))
    _epi_tensors(bias, (N,), aux, M, N)
    ws_bytes = _ws_bytes(workspace)
    _check("te_mxfp8_gemm_mxout", _lib.te_mxfp8_gemm_mxout(
        _ptr(a), _ptr(a_scale), _fmt(a_fmt), _ptr(b), _ptr(b_scale), _fmt(b_fmt), M, N, K,
        _ptr(d), _ptr(d_scale), _fmt(d_fmt), epi, _ptr(bias), _ptr(aux), _ptr(workspace), ws_bytes, _stream(stream)))


def te_mxfp8_grouped_gemm(m_splits, a, a_scale, a_fmt, b, b_scale, b_fmt, n: int, d, epilogue="none",
                          bias=None, aux=None, workspace=None, stream=None) -> None:
    _require(m_splits is not None and m_splits.dtype == torch.int32 and m_splits.dim() == 1,
             "m_splits: expected a 1-D int32 tensor (one row count per group)")
    G = m_splits.numel()
    total_m, _, K = _mx_operands(a, a_scale, b, b_scale)
    _require(b.shape[0] == G * int(n), f"b: expected {G} x {int(n)} = {G * int(n)} rows, got {b.shape[0]}")
    epi = _epilogue(epilogue)
    d_dtype = _gemm_out(d, "d", total_m, int(n), epi)
    _epi_tensors(bias, (G, int(n)), aux, total_m, int(n))
    ws_bytes = _ws_bytes(workspace)
    _check("te_mxfp8_grouped_gemm", _lib.te_mxfp8_grouped_gemm(
        m_splits.numel(), _ptr(m_splits), total_m, _ptr(a), _ptr(a_scale), _fmt(a_fmt), _ptr(b), _ptr(b_scale),
        _fmt(b_fmt), n, K, _ptr(d), d_dtype, epi, _ptr(bias), _ptr(aux), _ptr(workspace), ws_bytes,
        _stream(stream)))


def _block_scaling(mode) -> int:
    return BLOCK_SCALINGS[mode] if isinstance(mode, str) else int(mode)


def _block_scale_shape(rows, cols, block_2d):
    return ((rows + 127) // 128 if block_2d else rows, cols // 128)


def te_fp8_block_quantize(x, fmt, block_2d, q, scale_inv, stream=None) -> None:
    _require(x.dim() == 2, "x must be 2-D")
    rows, cols = x.shape
    _bf16(x, "x", (rows, cols))
    _codes(q, "q", (rows, cols))
    _f32(scale_inv, "scale_inv", _block_scale_shape(rows, cols, block_2d))
    _check("te_fp8_block_quantize", _lib.te_fp8_block_quantize(
        _ptr(x), rows, cols, _fmt(fmt), int(bool(block_2d)), _ptr(q), _ptr(scale_inv), _stream(stream)))


def te_fp8_block_scales_to_mx(scale_inv, rows: int, cols: int, block_2d: bool, mx_scale, stream=None) -> None:
    _f32(scale_inv, "scale_inv", _block_scale_shape(int(rows), int(cols), block_2d))
    _codes(mx_scale, "mx_scale", (int(rows), int(cols) // 32))
    _check("te_fp8_block_scales_to_mx", _lib.te_fp8_block_scales_to_mx(
        _ptr(scale_inv), int(rows), int(cols), int(bool(block_2d)), _ptr(mx_scale), _stream(stream)))


def te_fp8_block_gemm_workspace_size(M: int, N: int, K: int, mode="e8m0") -> int:
    return int(_lib.te_fp8_block_gemm_workspace_size(M, N, K, _block_scaling(mode)))


def te_fp8_block_gemm(a, a_scale_inv, a_fmt, b, b_scale_inv, b_fmt, b_block_2d, d, epilogue="none", bias=None,
                      aux=None, mode="e8m0", workspace=None, stream=None, beta=1.0) -> None:
    _require(a.dim() == 2 and b.dim() == 2, "a and b must be 2-D")
    M, K = a.shape
    N = b.shape[0]
    _codes(a, "a", (M, K))
    _codes(b, "b", (N, K))
    _f32(a_scale_inv, "a_scale_inv", _block_scale_shape(M, K, False))
    _f32(b_scale_inv, "b_scale_inv", _block_scale_shape(N, K, b_block_2d))
    epi = _epilogue(epilogue)
    d_dtype = _gemm_out(d, "d", M, N, epi, allow_fp16=True)
    _epi_tensors(bias, (N,), aux, M, N)
    ws_bytes = _ws_bytes(workspace)
    _check("te_fp8_block_gemm", _lib.te_fp8_block_gemm(
        _ptr(a), _ptr(a_scale_inv), _fmt(a_fmt), _ptr(b), _ptr(b_scale_inv), _fmt(b_fmt), int(bool(b_block_2d)),
        M, N, K, _ptr(d), d_dtype, epi, _ptr(bias), _ptr(aux), _block_scaling(mode), float(beta), _ptr(workspace),
        ws_bytes, _stream(stream)))


# -------------------------------------------- norms and gated feed-forward GEMMs

_NORM_DTYPES = {torch.bfloat16: TE_BF16, torch.float16: TE_FP16, torch.float32: TE_FP32}


try:  # the current stream's handle without building a Stream object (2.8 us of a small call's 11)
    from torch._C import _cuda_getCurrentRawStream as _current_stream
except ImportError:
    def _current_stream(index):
        return torch.cuda.current_stream(index).cuda_stream

try:  # the current device's index without the check that the GPU is in use (0.2 us)
    from torch._C import _cuda_getDevice as _current_device
except ImportError:
    _current_device = torch.cuda.current_device

_FLOATS = "bfloat16, float16 or float32"
_CODES = "1-byte codes (uint8)"
_B16 = "bf16 (or its int16 bits)"
_KINDS = {_CODES: frozenset(_BYTE_DTYPES), _B16: frozenset(_BF16_DTYPES), "float32": (torch.float32,),
          "int32": (torch.int32,), torch.bfloat16: (torch.bfloat16,), torch.float16: (torch.float16,),
          torch.float32: (torch.float32,)}


def _addr(t, name, shape, kind, index):
    """Device address of a required tensor: dense, of this shape and kind, on the call's device (the index of the
    first tensor's, -1 on the CPU)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.shape == shape and t.dtype in _KINDS[kind] and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in _KINDS[kind]:
        raise ValueError(f"{name}: expected {kind}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on the first tensor's device")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor (row-major, no strides)")
    return t.data_ptr()


def _opt(t, name, shape, kind, index):
    """Device address of an optional tensor (None stays None)."""
    return None if t is None else _addr(t, name, shape, kind, index)


def _workspace(t, index):
    """(address, bytes) of an optional workspace."""
    if t is None:
        return None, 0
    if t.get_device() != index:
        raise ValueError(f"workspace is on {t.device}, not on the first tensor's device")
    return _ptr(t), t.numel() * t.element_size()


def _index_of(t, name):
    _require(isinstance(t, torch.Tensor), f"{name} is required")
    _require(t.dim() == 2, f"{name} must be 2-D")
    return t.get_device()


def _run(name, args, index, stream):
    """The call with the tensors' device current, whatever the current one is, on `stream` or that device's current
    stream."""
    if index < 0:
        raise ValueError("expected a GPU tensor, got one on the CPU")
    handle = _current_stream(index) if stream is None else _stream(stream)
    if index == _current_device():
        status = _FNS[name](*args, handle)
    else:
        with torch.cuda.device(index):
            status = _FNS[name](*args, handle)
    if status != TE_OK:
        raise TemxError(name, status)


def _norm_args(kind, x, gamma):
    """(device index, kind, rows, cols, x's dtype code and dtype, gamma's dtype code and dtype)"""
    index = _index_of(x, "x")
    k = NORM_KINDS[kind] if isinstance(kind, str) else int(kind)
    xd = x.dtype
    _require(xd in _NORM_DTYPES, f"x: expected {_FLOATS}, got {xd}")
    _require(gamma is not None and (gamma.dtype == xd or gamma.dtype == torch.float32),
             "gamma: expected x's dtype or float32")
    rows, cols = x.shape
    return index, k, rows, cols, _NORM_DTYPES[xd], xd, _NORM_DTYPES[gamma.dtype], gamma.dtype


def te_norm_forward(kind, x, gamma, beta=None, eps=1e-5, y=None, q=None, q_scale=None, q_fmt="e4m3", residual=None,
                    sum_out=None, mean=None, rstd=None, stream=None) -> None:
    i, k, rows, cols, dt, xd, wdt, wd = _norm_args(kind, x, gamma)
    full, w = (rows, cols), (cols,)
    if q is not None:
        _require(cols % 32 == 0, "q: the MXFP8 output needs cols % 32 == 0")
    _run("te_norm_forward", (
        k, _addr(x, "x", full, xd, i), dt, rows, cols, _opt(residual, "residual", full, xd, i),
        _addr(gamma, "gamma", w, wd, i), _opt(beta, "beta", w, wd, i), wdt, eps, _opt(sum_out, "sum_out", full, xd, i),
        _opt(y, "y", full, xd, i), _opt(q, "q", full, _CODES, i),
        _opt(q_scale, "q_scale", (rows, cols // 32), _CODES, i), _fmt(q_fmt), _opt(mean, "mean", (rows,), "float32", i),
        _opt(rstd, "rstd", (rows,), "float32", i)), i, stream)


def te_norm_backward_workspace_size(rows: int, cols: int) -> int:
    return int(_lib.te_norm_backward_workspace_size(int(rows), int(cols)))


def te_norm_backward(kind, dy, x, gamma, mean, rstd, dx, dgamma, dbeta=None, dskip=None, workspace=None,
                     stream=None) -> None:
    i, k, rows, cols, dt, xd, wdt, wd = _norm_args(kind, x, gamma)
    full, w = (rows, cols), (cols,)
    ws, ws_bytes = _workspace(workspace, i)
    _run("te_norm_backward", (
        k, _addr(dy, "dy", full, xd, i), _addr(x, "x", full, xd, i), _opt(dskip, "dskip", full, xd, i), dt, rows, cols,
        _addr(gamma, "gamma", w, wd, i), wdt, _opt(mean, "mean", (rows,), "float32", i),
        _addr(rstd, "rstd", (rows,), "float32", i), _addr(dx, "dx", full, xd, i), _addr(dgamma, "dgamma", w, wd, i),
        _opt(dbeta, "dbeta", w, wd, i), ws, ws_bytes), i, stream)


def _activation(act) -> int:
    return ACTIVATIONS[act] if isinstance(act, str) else int(act)


def _gated_operands(i, a, a_scale, b, b_scale, rows_b):
    """Addresses of a [M, K], a_scale, b [rows_b, K] and b_scale."""
    M, K = a.shape
    return (_addr(a, "a", (M, K), _CODES, i), _addr(a_scale, "a_scale", (M, K // 32), _CODES, i),
            _addr(b, "b", (rows_b, K), _CODES, i), _addr(b_scale, "b_scale", (rows_b, K // 32), _CODES, i))


def te_mxfp8_gated_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(_lib.te_mxfp8_gated_gemm_workspace_size(M, N, K))


def te_mxfp8_gated_gemm(a, a_scale, a_fmt, b, b_scale, b_fmt, d, activation="silu", d_scale=None, d_fmt=None,
                        bias=None, aux=None, workspace=None, stream=None) -> None:
    """d_fmt None: d is bf16; "e4m3" / "e5m2": d is the MXFP8 operand (d, d_scale)."""
    i = _index_of(a, "a")
    _require(b is not None and b.dim() == 2, "b must be 2-D")
    M, K = a.shape
    _require(b.shape[0] % 2 == 0, "b: expected an even number of rows (gate rows, then up rows)")
    N = b.shape[0] // 2
    pa, psa, pb, psb = _gated_operands(i, a, a_scale, b, b_scale, 2 * N)
    if d_fmt is None:
        pd, pds, out = _addr(d, "d", (M, N), _B16, i), None, TE_BF16
        _require(d_scale is None, "d_scale: only with an MXFP8 d (d_fmt)")
    else:
        pd, out = _addr(d, "d", (M, N), _CODES, i), _fmt(d_fmt)
        pds = _addr(d_scale, "d_scale", (M, N // 32), _CODES, i)
    ws, ws_bytes = _workspace(workspace, i)
    _run("te_mxfp8_gated_gemm", (
        pa, psa, _fmt(a_fmt), pb, psb, _fmt(b_fmt), M, N, K, _activation(activation), pd, pds, out,
        _opt(bias, "bias", (2 * N,), _B16, i), _opt(aux, "aux", (M, 2 * N), _B16, i), ws, ws_bytes), i, stream)


def te_mxfp8_dgated_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(_lib.te_mxfp8_dgated_gemm_workspace_size(M, N, K))


def te_mxfp8_dgated_gemm(a, a_scale, a_fmt, b, b_scale, b_fmt, aux, d, activation="silu", workspace=None,
                         stream=None) -> None:
    i = _index_of(a, "a")
    _require(b is not None and b.dim() == 2, "b must be 2-D")
    M, K = a.shape
    N = b.shape[0]
    pa, psa, pb, psb = _gated_operands(i, a, a_scale, b, b_scale, N)
    ws, ws_bytes = _workspace(workspace, i)
    _run("te_mxfp8_dgated_gemm", (
        pa, psa, _fmt(a_fmt), pb, psb, _fmt(b_fmt), M, N, K, _activation(activation),
        _addr(aux, "aux", (M, 2 * N), _B16, i), _addr(d, "d", (M, 2 * N), _B16, i), ws, ws_bytes), i, stream)


def _groups(m_splits, i):
    """(count, address) of the splits."""
    _require(m_splits is not None and m_splits.dim() == 1, "m_splits: expected a 1-D int32 tensor")
    return m_splits.numel(), _addr(m_splits, "m_splits", m_splits.shape, "int32", i)


def te_mxfp8_grouped_gated_gemm(m_splits, a, a_scale, a_fmt, b, b_scale, b_fmt, n: int, d, activation="silu",
                                bias=None, aux=None, stream=None) -> None:
    i, n = _index_of(a, "a"), int(n)
    G, splits = _groups(m_splits, i)
    M, K = a.shape
    pa, psa, pb, psb = _gated_operands(i, a, a_scale, b, b_scale, G * 2 * n)
    _run("te_mxfp8_grouped_gated_gemm", (
        G, splits, M, pa, psa, _fmt(a_fmt), pb, psb, _fmt(b_fmt), n, K, _activation(activation),
        _addr(d, "d", (M, n), _B16, i), _opt(bias, "bias", (G, 2 * n), _B16, i),
        _opt(aux, "aux", (M, 2 * n), _B16, i)), i, stream)


def te_mxfp8_grouped_dgated_gemm(m_splits, a, a_scale, a_fmt, b, b_scale, b_fmt, n: int, aux, d, activation="silu",
                                 stream=None) -> None:
    i, n = _index_of(a, "a"), int(n)
    G, splits = _groups(m_splits, i)
    M, K = a.shape
    pa, psa, pb, psb = _gated_operands(i, a, a_scale, b, b_scale, G * n)
    _run("te_mxfp8_grouped_dgated_gemm", (
        G, splits, M, pa, psa, _fmt(a_fmt), pb, psb, _fmt(b_fmt), n, K, _activation(activation),
        _addr(aux, "aux", (M, 2 * n), _B16, i), _addr(d, "d", (M, 2 * n), _B16, i)), i, stream)


# ------------------------------------- the router, and tokens to their experts' rows and back

def _score(score) -> int:
    return SCORES[score] if isinstance(score, str) else int(score)


def _route_args(score, logits, experts):
    """(device index, score, logits' address and dtype, tokens, experts in all, topk, experts' address)"""
    index = _index_of(logits, "logits")
    dt = _NORM_DTYPES.get(logits.dtype)
    if dt is None:
        raise ValueError(f"logits: expected {_FLOATS}, got {logits.dtype}")
    if experts is None or experts.dim() != 2:
        raise ValueError("experts: expected a 2-D int32 tensor")
    tokens, n = shape = logits.shape
    topk = experts.shape[1]
    return (index, _score(score), _addr(logits, "logits", shape, logits.dtype, index), dt, tokens, n, topk,
            _addr(experts, "experts", (tokens, topk), "int32", index))


def te_moe_route(score, logits, experts, weights, bias=None, normalize=True, scale=1.0, stream=None) -> None:
    """experts int32 [tokens, topk] and weights float32 [tokens, topk] are written."""
    i, score, logits_at, dt, tokens, n, topk, experts_at = _route_args(score, logits, experts)
    _run("te_moe_route", (
        score, logits_at, dt, tokens, n, topk, None if bias is None else _addr(bias, "bias", (n,), "float32", i),
        1 if normalize else 0, scale, experts_at, _addr(weights, "weights", (tokens, topk), "float32", i)), i, stream)


def te_moe_route_backward(score, logits, experts, dweights, dlogits, normalize=True, scale=1.0, stream=None) -> None:
    i, score, logits_at, dt, tokens, n, topk, experts_at = _route_args(score, logits, experts)
    _run("te_moe_route_backward", (
        score, logits_at, dt, tokens, n, topk, 1 if normalize else 0, scale, experts_at,
        _addr(dweights, "dweights", (tokens, topk), "float32", i),
        _addr(dlogits, "dlogits", logits.shape, logits.dtype, i)), i, stream)


def te_moe_sort_workspace_size(slots: int, num_experts: int) -> int:
    return int(_lib.te_moe_sort_workspace_size(int(slots), int(num_experts)))


def te_moe_sort(experts, m_splits, row_of, slot_of, workspace=None, stream=None) -> None:
    """experts int32 of any shape (its slots in row-major order); row_of has its shape, slot_of its number of slots."""
    _require(isinstance(experts, torch.Tensor), "experts is required")
    i, shape, slots = experts.get_device(), experts.shape, experts.numel()
    G, splits = _groups(m_splits, i)
    ws, ws_bytes = _workspace(workspace, i)
    _run("te_moe_sort", (
        _addr(experts, "experts", shape, "int32", i), slots, G, splits, _addr(row_of, "row_of", shape, "int32", i),
        _addr(slot_of, "slot_of", (slots,), "int32", i), ws, ws_bytes), i, stream)


def _rows_args(row_of, tokens, index):
    """(topk, address) of row_of [tokens, topk]."""
    if row_of is None or row_of.dim() != 2:
        raise ValueError("row_of: expected a 2-D int32 tensor")
    topk = row_of.shape[1]
    return topk, _addr(row_of, "row_of", (tokens, topk), "int32", index)


def _rows_out(y, q, q_scale, dtype, cols, index, name):
    """(rows in all, addresses of y, q and q_scale) of the outputs with a row each slot."""
    first = y if y is not None else q
    if first is None:
        raise ValueError(f"{name} or q is required")
    if first.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    rows = first.shape[0]
    if q is None:
        if q_scale is not None:
            raise ValueError("q_scale: only with q")
        return rows, _addr(y, name, (rows, cols), dtype, index), None, None
    if cols % 32 != 0:
        raise ValueError("q: the MXFP8 output needs cols % 32 == 0")
    return (rows, _opt(y, name, (rows, cols), dtype, index), _addr(q, "q", (rows, cols), _CODES, index),
            _addr(q_scale, "q_scale", (rows, cols // 32), _CODES, index))


def _float_2d(t, name):
    """(device index, dtype, its code, shape) of a 2-D tensor of floats."""
    index = _index_of(t, name)
    dt = _NORM_DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name}: expected {_FLOATS}, got {t.dtype}")
    return index, t.dtype, dt, t.shape


def te_moe_dispatch(x, row_of, y=None, q=None, q_scale=None, q_fmt="e4m3", stream=None) -> None:
    i, xd, dt, shape = _float_2d(x, "x")
    tokens, cols = shape
    topk, row_at = _rows_args(row_of, tokens, i)
    rows, py, pq, pqs = _rows_out(y, q, q_scale, xd, cols, i, "y")
    _run("te_moe_dispatch", (_addr(x, "x", shape, xd, i), dt, tokens, cols, row_at, topk, rows, py, pq, pqs,
                             _fmt(q_fmt)), i, stream)


def te_moe_combine(rows, row_of, y, weights=None, stream=None) -> None:
    """weights None: all 1, the gradient of te_moe_dispatch."""
    i, xd, dt, shape = _float_2d(rows, "rows")
    total, cols = shape
    _require(y is not None and y.dim() == 2, "y: expected a 2-D tensor")
    tokens = y.shape[0]
    topk, row_at = _rows_args(row_of, tokens, i)
    _run("te_moe_combine", (_addr(rows, "rows", shape, xd, i), dt, total, cols, row_at,
                            _opt(weights, "weights", (tokens, topk), "float32", i), tokens, topk,
                            _addr(y, "y", (tokens, cols), xd, i)), i, stream)


def te_moe_combine_backward(dy, rows, row_of, weights, dweights, drows=None, q=None, q_scale=None, q_fmt="e5m2",
                            stream=None) -> None:
    i, xd, dt, shape = _float_2d(dy, "dy")
    tokens, cols = shape
    topk, row_at = _rows_args(row_of, tokens, i)
    total, pd, pq, pqs = _rows_out(drows, q, q_scale, xd, cols, i, "drows")
    _run("te_moe_combine_backward", (
        _addr(dy, "dy", shape, xd, i), _addr(rows, "rows", (total, cols), xd, i), dt, tokens, cols, row_at,
        _addr(weights, "weights", (tokens, topk), "float32", i), topk, total, pd, pq, pqs, _fmt(q_fmt),
        _addr(dweights, "dweights", (tokens, topk), "float32", i)), i, stream)


# ------------------------------------------------------ GEMMs with 4-bit weights

_W4_SCALES = {torch.bfloat16: TE_BF16, torch.float16: TE_FP16, torch.float32: TE_FP32, torch.uint8: TE_E8M0}
_W4_SCALES |= {getattr(torch, n): TE_E8M0 for n in ("float8_e8m0fnu",) if hasattr(torch, n)}
_KINDS["a scale type"] = frozenset(_W4_SCALES)


def _w4_args(x, w, w_fmt, w_scale, zero, rows, d, n):
    """(device index, the arguments up to the group size, M, K, d's address and dtype) of rows x K weights."""
    i = _index_of(x, "x")
    xd = x.dtype
    if xd is not torch.bfloat16 and xd is not torch.float16:
        raise ValueError(f"x: expected bfloat16 or float16, got {xd}")
    M, K = shape = x.shape
    if w_scale is None or w_scale.dim() != 2:
        raise ValueError("w_scale must be 2-D")
    scales = w_scale.shape[1]
    if K % 2 != 0 or (K % scales != 0 if scales else K != 0):
        raise ValueError(f"w_scale: {scales} columns do not divide K = {K} into groups")
    dt = _NORM_DTYPES[xd]
    scale_dt = _W4_SCALES.get(w_scale.dtype)
    if scale_dt is None or (scale_dt != dt and scale_dt != TE_FP32 and scale_dt != TE_E8M0):
        raise ValueError(f"w_scale: expected x's dtype, float32 or E8M0 codes (uint8), got {w_scale.dtype}")
    if d is None or (d.dtype != xd and d.dtype != torch.float32):
        raise ValueError("d: expected x's dtype or float32")
    args = (_addr(x, "x", shape, xd, i), dt, _addr(w, "w", (rows, K // 2), _CODES, i),
            W4_FORMATS[w_fmt] if isinstance(w_fmt, str) else int(w_fmt),
            _addr(w_scale, "w_scale", (rows, scales), "a scale type", i), scale_dt,
            None if zero is None else _addr(zero, "zero", (rows, scales), _CODES, i), K // scales if scales else 32)
    return i, args, M, K, _addr(d, "d", (M, n), d.dtype, i), _NORM_DTYPES[d.dtype]


def _rows_of(t, name, per=1):
    if t is None or t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.shape[0] % per != 0:
        raise ValueError(f"{name}: expected an even number of rows (gate rows, then up rows)")
    return t.shape[0] // per


def te_w4_gemm(x, w, w_fmt, w_scale, d, zero=None, bias=None, stream=None) -> None:
    """w uint8 [N, K/2] ("int4" or "e2m1" codes, even k in the low half), w_scale [N, groups of K], zero uint8 likewise."""
    N = _rows_of(w, "w")
    i, args, M, K, pd, dd = _w4_args(x, w, w_fmt, w_scale, zero, N, d, N)
    _run("te_w4_gemm", (*args, M, N, K, pd, dd, _opt(bias, "bias", (N,), x.dtype, i)), i, stream)


def te_w4_gated_gemm(x, w, w_fmt, w_scale, d, activation="silu", zero=None, bias=None, stream=None) -> None:
    N = _rows_of(w, "w", 2)
    i, args, M, K, pd, dd = _w4_args(x, w, w_fmt, w_scale, zero, 2 * N, d, N)
    _run("te_w4_gated_gemm", (*args, M, N, K, _activation(activation), pd, dd,
                              _opt(bias, "bias", (2 * N,), x.dtype, i)), i, stream)


def te_w4_grouped_gemm(m_splits, x, w, w_fmt, w_scale, n: int, d, zero=None, bias=None, stream=None) -> None:
    i, n = _index_of(x, "x"), int(n)
    G, splits = _groups(m_splits, i)
    _, args, M, K, pd, dd = _w4_args(x, w, w_fmt, w_scale, zero, G * n, d, n)
    _run("te_w4_grouped_gemm", (G, splits, M, *args, n, K, pd, dd, _opt(bias, "bias", (G, n), x.dtype, i)), i, stream)


def te_w4_grouped_gated_gemm(m_splits, x, w, w_fmt, w_scale, n: int, d, activation="silu", zero=None, bias=None,
                             stream=None) -> None:
    i, n = _index_of(x, "x"), int(n)
    G, splits = _groups(m_splits, i)
    _, args, M, K, pd, dd = _w4_args(x, w, w_fmt, w_scale, zero, G * 2 * n, d, n)
    _run("te_w4_grouped_gated_gemm", (G, splits, M, *args, n, K, _activation(activation), pd, dd,
                                      _opt(bias, "bias", (G, 2 * n), x.dtype, i)), i, stream)


# ------------------------------------------------------- allocating helpers

def mxfp8_quantize(x, fmt="e4m3", direction="row", stream=None):
    """bf16 [rows, cols] (torch.bfloat16 or int16/uint16 bits) -> (q_row, s_row, q_col, s_col), None where
    a direction is not requested."""
    rows, cols = x.shape
    d = DIRECTIONS[direction]
    dev = x.device
    q_row = s_row = q_col = s_col = None
    if d & TE_ROWWISE:
        q_row = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        s_row = torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev)
    if d & TE_COLWISE:
        q_col = torch.empty((cols, rows), dtype=torch.uint8, device=dev)
        s_col = torch.empty((cols, rows // 32), dtype=torch.uint8, device=dev)
    te_mxfp8_quantize(x, fmt, d, q_row, s_row, q_col, s_col, stream)
    return q_row, s_row, q_col, s_col


def mxfp8_quantize_bgrad(x, fmt="e5m2", bgrad_dtype=torch.float32, stream=None):
    """bf16 [rows, cols] output gradient -> (q_row, s_row, q_col, s_col, bgrad), one pass; bgrad [cols] is
    the column sum of x (fp32 accumulation), as float32 or bfloat16."""
    rows, cols = x.shape
    dev = x.device
    q_row = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    s_row = torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev)
    q_col = torch.empty((cols, rows), dtype=torch.uint8, device=dev)
    s_col = torch.empty((cols, rows // 32), dtype=torch.uint8, device=dev)
    bgrad = torch.empty(cols, dtype=bgrad_dtype, device=dev)
    ws = torch.empty(max(te_mxfp8_quantize_bgrad_workspace_size(rows, cols), 16), dtype=torch.uint8, device=dev)
    te_mxfp8_quantize_bgrad(x, fmt, q_row, s_row, q_col, s_col, bgrad, ws, stream)
    return q_row, s_row, q_col, s_col, bgrad


class DelayedScaling:
    """Device state of one tensor under delayed scaling: scale (starts at 1) and the amax history
    (zeros, newest first).  step(x) casts x with the current scale and updates the state."""

    def __init__(self, fmt="e4m3", history_len=16, algo="max", margin=0, device="cuda"):
        self.fmt, self.algo, self.margin = fmt, algo, margin
        self.scale = torch.ones(1, dtype=torch.float32, device=device)
        self.history = torch.zeros(history_len, dtype=torch.float32, device=device)

    def step(self, x, stream=None):
        """-> (q, q_scale_inv): x cast with the scale as it stood, and that scale's inverse."""
        dev = x.device
        q = torch.empty(x.shape, dtype=torch.uint8, device=dev)
        q_inv = torch.empty(1, dtype=torch.float32, device=dev)
        ws = torch.empty(max(te_amax_workspace_size(x.numel()), 4), dtype=torch.uint8, device=dev)
        te_fp8_cast_delayed_scaling(x, self.fmt, q, q_inv, self.scale, self.history, ws, self.algo, self.margin,
                                    stream)
        return q, q_inv


def fp8_gemm(a, a_scale_inv, a_fmt, b, b_scale_inv, b_fmt, epilogue="none", bias=None, out_dtype=torch.bfloat16,
             stream=None):
    """Per-tensor FP8 GEMM -> (D, aux)."""
    M, N = a.shape[0], b.shape[0]
    d = torch.empty((M, N), dtype=out_dtype, device=a.device)
    aux = torch.empty((M, N), dtype=torch.bfloat16, device=a.device) if epilogue == "bias_gelu_aux" else None
    te_fp8_gemm(a, a_scale_inv, a_fmt, b, b_scale_inv, b_fmt, d, epilogue, bias, aux, None, stream)
    return d, aux


def amax(x, stream=None):
    ws = torch.empty(max(te_amax_workspace_size(x.numel()), 4), dtype=torch.uint8, device=x.device)
    out = torch.empty(1, dtype=torch.float32, device=x.device)
    te_amax_reduce(x, out, ws, stream)
    return out


def fp8_cast_current_scaling(x, fmt="e4m3", stream=None):
    """-> (q, amax, scale, scale_inv) with q shaped like x."""
    dev = x.device
    ws = torch.empty(max(te_amax_workspace_size(x.numel()), 4), dtype=torch.uint8, device=dev)
    q = torch.empty(x.shape, dtype=torch.uint8, device=dev)
    a, s, si = (torch.empty(1, dtype=torch.float32, device=dev) for _ in range(3))
    te_fp8_cast_current_scaling(x, fmt, q, a, s, si, ws, stream)
    return q, a, s, si


def gemm_workspace(M: int, N: int, K: int, device="cuda"):
    """The workspace te_mxfp8_gemm / te_mxfp8_gemm_mxout use for an M x N x K GEMM (None if none)."""
    n = te_mxfp8_gemm_workspace_size(M, N, K)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def mxfp8_gemm(a, a_scale, a_fmt, b, b_scale, b_fmt, epilogue="none", bias=None, out_dtype=torch.bfloat16,
               aux=None, out=None, stream=None, workspace="auto"):
    """-> (D, aux) for D = epilogue(A . B^T).  aux is written and returned for "bias_gelu_aux" and is
    the saved pre-activation read by "dgelu"; "accumulate" adds into the given fp32 ``out``.
    workspace: "auto" allocates what the GEMM can use, or a tensor, or None for none."""
    M, N = a.shape[0], b.shape[0]
    d = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=a.device)
    if epilogue == "bias_gelu_aux":
        aux = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    if isinstance(workspace, str):
        workspace = gemm_workspace(M, N, a.shape[1], a.device)
    te_mxfp8_gemm(a, a_scale, a_fmt, b, b_scale, b_fmt, d, epilogue, bias, aux, workspace, stream)
    return d, (aux if epilogue == "bias_gelu_aux" else None)


def mxfp8_gemm_mxout(a, a_scale, a_fmt, b, b_scale, b_fmt, epilogue="none", bias=None, out_fmt="e4m3",
                     stream=None):
    """-> (codes, scales, aux): D = epilogue(A . B^T) as a rowwise MXFP8 operand (codes [M, N], E8M0
    scales [M, N/32]); aux as mxfp8_gemm."""
    M, N = a.shape[0], b.shape[0]
    d = torch.empty((M, N), dtype=torch.uint8, device=a.device)
    ds = torch.empty((M, N // 32), dtype=torch.uint8, device=a.device)
    aux = torch.empty((M, N), dtype=torch.bfloat16, device=a.device) if epilogue == "bias_gelu_aux" else None
    te_mxfp8_gemm_mxout(a, a_scale, a_fmt, b, b_scale, b_fmt, d, ds, out_fmt, epilogue, bias, aux,
                        gemm_workspace(M, N, a.shape[1], a.device), stream)
    return d, ds, aux


def mxfp8_grouped_gemm(m_splits, a, a_scale, a_fmt, b, b_scale, b_fmt, n, epilogue="none", bias=None,
                       out_dtype=torch.bfloat16, aux=None, out=None, stream=None):
    total_m = a.shape[0]
    d = out if out is not None else torch.empty((total_m, n), dtype=out_dtype, device=a.device)
    if epilogue == "bias_gelu_aux":
        aux = torch.empty((total_m, n), dtype=torch.bfloat16, device=a.device)
    te_mxfp8_grouped_gemm(m_splits, a, a_scale, a_fmt, b, b_scale, b_fmt, n, d, epilogue, bias, aux, None, stream)
    return d, (aux if epilogue == "bias_gelu_aux" else None)


def fp8_block_quantize(x, fmt="e4m3", block_2d=False, stream=None):
    """bf16 [rows, cols] -> (codes uint8 [rows, cols], scale_inv float [rows or ceil(rows/128), cols/128])."""
    rows, cols = x.shape
    q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    srows = (rows + 127) // 128 if block_2d else rows
    s = torch.empty((srows, cols // 128), dtype=torch.float32, device=x.device)
    te_fp8_block_quantize(x, fmt, block_2d, q, s, stream)
    return q, s


def fp8_block_scales_to_mx(scale_inv, rows: int, cols: int, block_2d: bool, stream=None):
    """FP32 block scale inverses -> E8M0 MXFP8 scales uint8 [rows, cols/32]."""
    out = torch.empty((rows, cols // 32), dtype=torch.uint8, device=scale_inv.device)
    te_fp8_block_scales_to_mx(scale_inv, rows, cols, block_2d, out, stream)
    return out


def fp8_block_gemm(a, a_scale_inv, a_fmt, b, b_scale_inv, b_fmt, b_block_2d=True, epilogue="none", bias=None,
                   out_dtype=torch.bfloat16, aux=None, out=None, mode="e8m0", workspace=None, stream=None, beta=1.0):
    """Blockwise FP8 GEMM -> (D, aux); scale inverses float [M, K/128] for A and [N, K/128] (1-D) or
    [ceil(N/128), K/128] (2-D) for B; mode "e8m0" (scales cast to powers of two) or "fp32"; D bf16, fp16
    or fp32; "accumulate" adds into the fp32 ``out`` scaled by ``beta``."""
    M, K = a.shape
    N = b.shape[0]
    d = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=a.device)
    if epilogue == "bias_gelu_aux":
        aux = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    if workspace is None:
        ws_bytes = te_fp8_block_gemm_workspace_size(M, N, K, mode)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=a.device) if ws_bytes else None
    te_fp8_block_gemm(a, a_scale_inv, a_fmt, b, b_scale_inv, b_fmt, b_block_2d, d, epilogue, bias, aux, mode,
                      workspace, stream, beta)
    return d, (aux if epilogue == "bias_gelu_aux" else None)


def _allocating_on(stream, device):
    """Context in which a helper's outputs and workspaces belong to the stream that its call runs on (memory freed by
    the caller is then reused in that stream's order)."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def norm_forward(kind, x, gamma, beta=None, eps=1e-5, residual=None, mx_fmt=None, want_y=True, stream=None):
    """Layer norm ("layer") or RMS norm ("rms") of x [rows, cols] (+ residual) ->
    (y, q, q_scale, sum, mean, rstd): y in x's dtype (None if not wanted), its MXFP8 operand with mx_fmt, the sum
    with a residual (what norm_backward takes as x), the statistics (mean None for RMS norm)."""
    rows, cols = x.shape
    dev = x.device
    with _allocating_on(stream, dev):
        y = torch.empty_like(x) if want_y else None
        q = torch.empty((rows, cols), dtype=torch.uint8, device=dev) if mx_fmt else None
        qs = torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev) if mx_fmt else None
        total = torch.empty_like(x) if residual is not None else None
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        mean = torch.empty_like(rstd) if NORM_KINDS[kind] == TE_NORM_LAYER else None
        te_norm_forward(kind, x, gamma, beta, eps, y, q, qs, mx_fmt or "e4m3", residual, total, mean, rstd, stream)
    return y, q, qs, total, mean, rstd


def norm_backward(kind, dy, x, gamma, mean, rstd, dskip=None, want_dbeta=True, stream=None):
    """-> (dx, dgamma, dbeta): dx + dskip where given; dbeta None for RMS norm or where not wanted."""
    dev = x.device
    with _allocating_on(stream, dev):
        dx, dgamma = torch.empty_like(x), torch.empty_like(gamma)
        dbeta = torch.empty_like(gamma) if want_dbeta and NORM_KINDS[kind] == TE_NORM_LAYER else None
        size = te_norm_backward_workspace_size(*x.shape)
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        te_norm_backward(kind, dy, x, gamma, mean, rstd, dx, dgamma, dbeta, dskip, ws, stream)
    return dx, dgamma, dbeta


def mxfp8_gated_gemm(a, a_scale, a_fmt, b, b_scale, b_fmt, activation="silu", bias=None, out_fmt=None, want_aux=False,
                     stream=None):
    """act(A Wg^T + bg) * (A Wu^T + bu) with b = [Wg; Wu] -> (D, d_scale, aux): D bf16, or with out_fmt MXFP8 codes
    and their E8M0 scales; aux, the bf16 pre-activations [gate | up] that mxfp8_dgated_gemm takes, where wanted."""
    M, N, K = a.shape[0], b.shape[0] // 2, a.shape[1]
    dev = a.device
    with _allocating_on(stream, dev):
        d = torch.empty((M, N), dtype=torch.uint8 if out_fmt else torch.bfloat16, device=dev)
        ds = torch.empty((M, N // 32), dtype=torch.uint8, device=dev) if out_fmt else None
        aux = torch.empty((M, 2 * N), dtype=torch.bfloat16, device=dev) if want_aux else None
        size = te_mxfp8_gated_gemm_workspace_size(M, N, K)
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        te_mxfp8_gated_gemm(a, a_scale, a_fmt, b, b_scale, b_fmt, d, activation, ds, out_fmt, bias, aux, ws, stream)
    return d, ds, aux


def mxfp8_dgated_gemm(a, a_scale, a_fmt, b, b_scale, b_fmt, aux, activation="silu", stream=None):
    """[dgate | dup] bf16 [M, 2N] from the output gradient's GEMM A . B^T and the saved pre-activations aux."""
    M, N, K = a.shape[0], b.shape[0], a.shape[1]
    with _allocating_on(stream, a.device):
        d = torch.empty((M, 2 * N), dtype=torch.bfloat16, device=a.device)
        size = te_mxfp8_dgated_gemm_workspace_size(M, N, K)
        ws = torch.empty(size, dtype=torch.uint8, device=a.device) if size else None
        te_mxfp8_dgated_gemm(a, a_scale, a_fmt, b, b_scale, b_fmt, aux, d, activation, ws, stream)
    return d


def moe_route(score, logits, topk, bias=None, normalize=True, scale=1.0, stream=None):
    """The router ("softmax" or "sigmoid" scores) -> (experts int32 [tokens, topk], weights float32 [tokens, topk])."""
    with _allocating_on(stream, logits.device):
        experts = torch.empty((logits.shape[0], topk), dtype=torch.int32, device=logits.device)
        weights = torch.empty((logits.shape[0], topk), dtype=torch.float32, device=logits.device)
        te_moe_route(score, logits, experts, weights, bias, normalize, scale, stream)
    return experts, weights


def moe_route_backward(score, logits, experts, dweights, normalize=True, scale=1.0, stream=None):
    """-> dlogits, the gradient of the logits from moe_route's weights' one."""
    with _allocating_on(stream, logits.device):
        dlogits = torch.empty_like(logits)
        te_moe_route_backward(score, logits, experts, dweights, dlogits, normalize, scale, stream)
    return dlogits


def moe_sort(experts, num_experts: int, stream=None):
    """experts int32 [tokens, topk] -> (m_splits [num_experts], row_of [tokens, topk], slot_of [tokens * topk])."""
    dev = experts.device
    with _allocating_on(stream, dev):
        m_splits = torch.empty(num_experts, dtype=torch.int32, device=dev)
        row_of = torch.empty_like(experts)
        slot_of = torch.empty(experts.numel(), dtype=torch.int32, device=dev)
        size = te_moe_sort_workspace_size(experts.numel(), num_experts)
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        te_moe_sort(experts, m_splits, row_of, slot_of, ws, stream)
    return m_splits, row_of, slot_of


def moe_dispatch(x, row_of, mx_fmt=None, want_y=True, stream=None):
    """Each token's row at its slots' rows -> (y, q, q_scale) with tokens * topk rows: y in x's dtype (None if not
    wanted), the MXFP8 operand with mx_fmt.  Rows behind the last are unset."""
    rows, cols, dev = row_of.numel(), x.shape[1], x.device
    with _allocating_on(stream, dev):
        y = torch.empty((rows, cols), dtype=x.dtype, device=dev) if want_y else None
        q = torch.empty((rows, cols), dtype=torch.uint8, device=dev) if mx_fmt else None
        qs = torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev) if mx_fmt else None
        te_moe_dispatch(x, row_of, y, q, qs, mx_fmt or "e4m3", stream)
    return y, q, qs


def moe_combine(rows, row_of, weights=None, stream=None):
    """-> y [tokens, cols], each token's rows added up with its weights (None: all 1, the gradient of moe_dispatch)."""
    with _allocating_on(stream, rows.device):
        y = torch.empty((row_of.shape[0], rows.shape[1]), dtype=rows.dtype, device=rows.device)
        te_moe_combine(rows, row_of, y, weights, stream)
    return y


def moe_combine_backward(dy, rows, row_of, weights, mx_fmt=None, want_drows=True, stream=None):
    """-> (drows, dweights, q, q_scale): drows in dy's dtype (None if not wanted), its MXFP8 operand with mx_fmt.  Rows
    behind the last are unset."""
    total, cols, dev = rows.shape[0], rows.shape[1], rows.device
    with _allocating_on(stream, dev):
        drows = torch.empty_like(rows) if want_drows else None
        q = torch.empty((total, cols), dtype=torch.uint8, device=dev) if mx_fmt else None
        qs = torch.empty((total, cols // 32), dtype=torch.uint8, device=dev) if mx_fmt else None
        dweights = torch.empty_like(weights)
        te_moe_combine_backward(dy, rows, row_of, weights, dweights, drows, q, qs, mx_fmt or "e5m2", stream)
    return drows, dweights, q, qs


def w4_gemm(x, w, w_fmt, w_scale, zero=None, bias=None, activation=None, m_splits=None, out_dtype=None, stream=None):
    """x W^T of 4-bit weights (te_w4_gemm); with an activation the gated form (w = [gate rows; up rows]), with m_splits
    the grouped one (the experts' weights stacked) -> D in x's dtype or out_dtype."""
    M, dev = x.shape[0], x.device
    per = (m_splits.numel() if m_splits is not None else 1) * (2 if activation else 1)
    n = w.shape[0] // per
    with _allocating_on(stream, dev):
        d = torch.empty((M, n), dtype=out_dtype or x.dtype, device=dev)
        more = {"zero": zero, "bias": bias, "stream": stream}
        if m_splits is not None and activation:
            te_w4_grouped_gated_gemm(m_splits, x, w, w_fmt, w_scale, n, d, activation, **more)
        elif m_splits is not None:
            te_w4_grouped_gemm(m_splits, x, w, w_fmt, w_scale, n, d, **more)
        elif activation:
            te_w4_gated_gemm(x, w, w_fmt, w_scale, d, activation, **more)
        else:
            te_w4_gemm(x, w, w_fmt, w_scale, d, **more)
    return d
