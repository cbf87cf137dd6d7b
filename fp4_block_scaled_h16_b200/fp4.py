"""ctypes binding of libfp4.so (C ABI in include/fp4.h).

Argument marshalling only: every step of quantization and GEMM runs in the
library's CUDA kernels.  Pointer arguments take a torch tensor (its
``data_ptr()``), an integer address or None; ``stream`` defaults to torch's
current CUDA stream, and what a helper allocates comes from the memory of the
stream that it runs on.  A non-OK status raises :class:`Fp4Error`.

Importing this module loads the library and raises ImportError if it has not
been built (``python -m fp4_block_scaled_h16_b200.build``): there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libfp4.so is not built: run `python -m fp4_block_scaled_h16_b200.build`")

_lib = ctypes.CDLL(LIB_PATH)

# enums (include/fp4.h)
FP4_OK, FP4_ERR_INVALID_ARG, FP4_ERR_UNSUPPORTED_SHAPE, FP4_ERR_MISALIGNED = 0, 1, 2, 3
FP4_ERR_WORKSPACE, FP4_ERR_NO_DEVICE, FP4_ERR_CUDA, FP4_ERR_TIMEOUT, FP4_ERR_UNSUPPORTED = 4, 5, 6, 7, 8
FP4_MXFP4, FP4_NVFP4, FP4_UFP4 = 0, 1, 2
FP4_RTNE, FP4_SR = 0, 1
FP4_ROT_NONE, FP4_ROT_H16, FP4_ROT_H32, FP4_ROT_RH16, FP4_ROT_RH32 = 0, 1, 2, 3, 4
FP4_IN_F32, FP4_IN_BF16 = 0, 1
FP4_OUT_F32, FP4_OUT_BF16 = 0, 1

EXPORTS = ("fp4_scales_bytes", "fp4_quantize_workspace_size", "fp4_amax", "fp4_quantize",
           "fp4_gemm", "fp4_last_error", "fp4_status_string", "fp4_set_wait_limit",
           "fp4_quantize_noalloc", "fp4_requantize", "fp4_rotate", "fp4_mxnorm_quantize",
           "fp4_gemm_workspace_size", "fp4_channel_amax", "fp4_outctl_workspace_size", "fp4_outctl_quantize",
           "fp4_gemm_outctl", "fp4_set_gemm_cta_pairs", "fp4_quantize_both_axes", "fp4_fp8_block_scales_count",
           "fp4_fp8_block_quantize", "fp4_fp8_block_gemm", "fp4_norm_residual",
           "fp4_norm_residual_backward_workspace_size", "fp4_norm_residual_backward")

_P, _I, _I64, _U64, _U32, _SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64,
                                 ctypes.c_uint32, ctypes.c_size_t)
_lib.fp4_status_string.argtypes = [_I]
_lib.fp4_status_string.restype = ctypes.c_char_p
_lib.fp4_scales_bytes.argtypes = [_I64, _I64, _I]
_lib.fp4_scales_bytes.restype = _SZ
_lib.fp4_quantize_workspace_size.argtypes = [_I, _I, _I, ctypes.POINTER(_SZ)]
_lib.fp4_amax.argtypes = [_P, _I, _I64, _I64, _I64, _I, _I, _U64, _P, _P]
_lib.fp4_quantize.argtypes = [_P, _I, _I64, _I64, _I64, _I, _I, _I, _I, _I, _U64, _U32, _P,
                              _P, _P, _P, _P, _P, _SZ, _P]
_lib.fp4_quantize_both_axes.argtypes = [_P, _I, _I64, _I64, _I64, _I, _I, _U64, _I, _U32, _P, _P, _P, _I, _U32, _P,
                                        _P, _P, _P, _SZ, _P]
_lib.fp4_quantize_noalloc.argtypes = [_P, _I, _I64, _I64, _I64, _I, _I, _I, _I, _U64, _U32, _P, _P, _P, _P]
_lib.fp4_requantize.argtypes = [_P, _P, _P, _P, _I64, _I64, _I, _I, _I, _I, _I, _I, _U64, _U32, _P, _P, _P, _P, _P,
                                _P, _SZ, _P]
_lib.fp4_mxnorm_quantize.argtypes = [_P, _I, _I64, _I64, _I64, _I, _I, _I, ctypes.c_float, _U64, _U32, _P, _P, _P,
                                     _P, _P, _SZ, _P]
_lib.fp4_channel_amax.argtypes = [_P, _I, _I64, _I64, _I64, _P, _P]
_lib.fp4_outctl_workspace_size.argtypes = [_I64, ctypes.POINTER(_SZ)]
_lib.fp4_outctl_quantize.argtypes = [_P, _I, _I64, _I64, _I64, _P, _I64, _I64, _I, _I, _U64, _U32, _P, _P, _P, _P, _P,
                                     _P, _SZ, _P]
_lib.fp4_gemm_outctl.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _I, _I64, _P]
_lib.fp4_rotate.argtypes = [_P, _I, _I64, _I64, _I64, _I, _I, _U64, _P, _I64, _P]
_lib.fp4_gemm.argtypes = [_I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _I, _I64, _P, _SZ, _P]
_lib.fp4_gemm_workspace_size.argtypes = [_I, _I, _I64, _I64, _I64, ctypes.POINTER(_SZ)]
_F = ctypes.c_float
_lib.fp4_fp8_block_scales_count.argtypes = [_I64, _I64, _I]
_lib.fp4_fp8_block_scales_count.restype = _SZ
_lib.fp4_fp8_block_quantize.argtypes = [_P, _I, _I64, _I64, _I64, _I, _P, _I64, _P, _P, _I64, _P, _P]
_lib.fp4_fp8_block_gemm.argtypes = [_P, _I64, _P, _P, _I64, _P, _I, _I64, _I64, _I64, _P, _I, _I64, _P]
_lib.fp4_norm_residual.argtypes = [_P, _I64, _P, _I64, _I, _I64, _I64, _P, _P, _I64, _I64, _F, _P, _F, _P, _I64, _P,
                                   _I64, _P, _I64, _P, _P, _P, _P]
_lib.fp4_norm_residual_backward_workspace_size.argtypes = [_I64, _I64, _I, _I, _I, _I64, ctypes.POINTER(_SZ)]
_lib.fp4_norm_residual_backward.argtypes = [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _I, _I64, _I64, _P, _P, _I64, _I64,
                                            _F, _P, _P, _P, _P, _I64, _P, _I64, _P, _P, _P, _P, _SZ, _P]
_lib.fp4_last_error.argtypes = [_P]
_lib.fp4_set_wait_limit.argtypes = [_U32]
_lib.fp4_set_wait_limit.restype = None
_lib.fp4_set_gemm_cta_pairs.argtypes = [_I]
_lib.fp4_set_gemm_cta_pairs.restype = None
for _f in ("fp4_amax", "fp4_rotate", "fp4_mxnorm_quantize", "fp4_gemm_workspace_size", "fp4_channel_amax",
           "fp4_outctl_workspace_size", "fp4_outctl_quantize", "fp4_gemm_outctl", "fp4_quantize", "fp4_quantize_noalloc",
           "fp4_quantize_both_axes", "fp4_requantize", "fp4_gemm", "fp4_last_error",
           "fp4_quantize_workspace_size", "fp4_fp8_block_quantize", "fp4_fp8_block_gemm", "fp4_norm_residual",
           "fp4_norm_residual_backward_workspace_size", "fp4_norm_residual_backward"):
    getattr(_lib, _f).restype = _I


class Fp4Error(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = status
        super().__init__("%s%s" % (where + ": " if where else "", fp4_status_string(status)))


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on_stream(helper):
    """Make the helper's `stream` torch's current one for the call.  Memory from
    another stream's pool may still be in use there, and goes back to that pool
    while the call on `stream` may not have run yet."""
    at = list(inspect.signature(helper).parameters).index("stream")

    @functools.wraps(helper)
    def call(*args, **kwargs):
        stream = args[at] if len(args) > at else kwargs.get("stream")
        if stream is None:
            return helper(*args, **kwargs)
        import torch
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(_stream(stream))
        if stream.device_index != torch.cuda.current_device():
            raise ValueError("stream is on %s, the current device is cuda:%d" % (stream.device, torch.cuda.current_device()))
        with torch.cuda.stream(stream):
            return helper(*args, **kwargs)
    return call


def _check(status: int, where: str):
    if status != FP4_OK:
        raise Fp4Error(status, where)


def fp4_status_string(status: int) -> str:
    return _lib.fp4_status_string(status).decode()


def fp4_scales_bytes(lines: int, K: int, fmt: int) -> int:
    return _lib.fp4_scales_bytes(lines, K, fmt)


def fp4_quantize_workspace_size(fmt: int, double_block: bool, amax_given: bool) -> int:
    n = _SZ(0)
    _check(_lib.fp4_quantize_workspace_size(fmt, int(double_block), int(amax_given), ctypes.byref(n)),
           "fp4_quantize_workspace_size")
    return n.value


def fp4_set_wait_limit(polls: int) -> None:
    _lib.fp4_set_wait_limit(polls)


def fp4_set_gemm_cta_pairs(enable: bool) -> None:
    _lib.fp4_set_gemm_cta_pairs(int(bool(enable)))


def fp4_amax(x, in_dtype, rows, cols, ld, rotation, axis, seed, amax_out, stream=None) -> None:
    _check(_lib.fp4_amax(_ptr(x), in_dtype, rows, cols, ld, rotation, axis, seed, _ptr(amax_out),
                         _stream(stream)), "fp4_amax")


def fp4_rotate(x, in_dtype, rows, cols, ld, rotation, axis, seed, y, ldy, stream=None) -> None:
    _check(_lib.fp4_rotate(_ptr(x), in_dtype, rows, cols, ld, rotation, axis, seed, _ptr(y), ldy,
                           _stream(stream)), "fp4_rotate")


@_on_stream
def rotate(x, rotation, seed=0, out=None, stream=None):
    """The rotation alone along the rows of a 2-D CUDA tensor, in its own dtype (fp4_rotate)."""
    import torch
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else cols
    y = out if out is not None else torch.empty((rows, cols), dtype=x.dtype, device=x.device)
    fp4_rotate(x, in_dtype_of(x), rows, cols, ld, rotation, 1, seed, y, y.stride(0) if rows > 1 else cols, stream)
    return y


def fp4_mxnorm_quantize(x, in_dtype, rows, cols, ld, fmt, rounding, p, c, seed, tensor_id, codes, scales,
                        tensor_scale, rho, workspace, workspace_bytes, stream=None) -> None:
    _check(_lib.fp4_mxnorm_quantize(_ptr(x), in_dtype, rows, cols, ld, fmt, rounding, p, c, seed, tensor_id,
                                    _ptr(codes), _ptr(scales), _ptr(tensor_scale), _ptr(rho), _ptr(workspace),
                                    workspace_bytes, _stream(stream)), "fp4_mxnorm_quantize")


@_on_stream
def mxnorm_quantize(x, fmt, p, c, rounding=FP4_RTNE, seed=0, tensor_id=0, out=None, rho=None, workspace=None,
                    stream=None):
    """MXNorm fused with the cast of a 2-D CUDA tensor along its rows
    (fp4_mxnorm_quantize): returns the quantized tensor with its "rho" [rows]."""
    import torch
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else cols
    q = out if out is not None else alloc_qtensor(rows, cols, fmt, False, x.device)
    r = rho if rho is not None else torch.empty(max(rows, 1), dtype=torch.float32, device=x.device)
    ws_bytes = 0 if fmt == FP4_MXFP4 else 256
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    fp4_mxnorm_quantize(x, in_dtype_of(x), rows, cols, ld, fmt, rounding, p, c, seed, tensor_id, q["codes"],
                        q["scales"], q["tensor_scale"], r, workspace if ws_bytes else None, ws_bytes, stream)
    q["rho"] = r
    return q


def fp4_quantize(x, in_dtype, rows, cols, ld, fmt, rounding, rotation, axis, double_block, seed,
                 tensor_id, tensor_amax, codes, scales, outer_scales, tensor_scale, workspace,
                 workspace_bytes, stream=None) -> None:
    _check(_lib.fp4_quantize(_ptr(x), in_dtype, rows, cols, ld, fmt, rounding, rotation, axis,
                             int(double_block), seed, tensor_id, _ptr(tensor_amax), _ptr(codes),
                             _ptr(scales), _ptr(outer_scales), _ptr(tensor_scale), _ptr(workspace),
                             workspace_bytes, _stream(stream)), "fp4_quantize")


def fp4_requantize(src_codes, src_scales, src_outer, src_tensor_scale, lines, K, src_fmt, src_double_block,
                   fmt, rounding, rotation, double_block, seed, tensor_id, tensor_amax, codes, scales,
                   outer_scales, tensor_scale, workspace, workspace_bytes, stream=None) -> None:
    _check(_lib.fp4_requantize(_ptr(src_codes), _ptr(src_scales), _ptr(src_outer), _ptr(src_tensor_scale),
                               lines, K, src_fmt, int(src_double_block), fmt, rounding, rotation,
                               int(double_block), seed, tensor_id, _ptr(tensor_amax), _ptr(codes), _ptr(scales),
                               _ptr(outer_scales), _ptr(tensor_scale), _ptr(workspace), workspace_bytes,
                               _stream(stream)), "fp4_requantize")


@_on_stream
def requantize(q, fmt, rounding=FP4_RTNE, rotation=FP4_ROT_NONE, double_block=False, seed=0, tensor_id=0,
               tensor_amax=None, out=None, workspace=None, stream=None):
    """Re-quantize the quantized tensor q (lines x K) along the other axis: the
    result has K lines of q["lines"] elements (fp4_requantize)."""
    import torch
    lines, K = q["lines"], q["K"]
    r = out if out is not None else alloc_qtensor(K, lines, fmt, double_block, q["codes"].device)
    ws_bytes = fp4_quantize_workspace_size(fmt, double_block, tensor_amax is not None)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q["codes"].device)
    fp4_requantize(q["codes"], q["scales"], q["outer"], q["tensor_scale"] if q["format"] != FP4_MXFP4 else None,
                   lines, K, q["format"], q["double_block"], fmt, rounding, rotation, double_block, seed,
                   tensor_id, tensor_amax, r["codes"], r["scales"], r["outer"], r["tensor_scale"],
                   workspace if ws_bytes else None, ws_bytes, stream)
    return r


def fp4_quantize_noalloc(x, in_dtype, rows, cols, ld, fmt, rounding, rotation, axis, seed, tensor_id,
                         codes, scales, tensor_scale, stream=None) -> None:
    """fp4_quantize (NVFP4 / UFP4, internal amax) without a workspace: the
    scratch is the library's static device array.  For callers that cannot
    allocate device memory; concurrent calls race on that array."""
    _check(_lib.fp4_quantize_noalloc(_ptr(x), in_dtype, rows, cols, ld, fmt, rounding, rotation, axis, seed,
                                     tensor_id, _ptr(codes), _ptr(scales), _ptr(tensor_scale), _stream(stream)),
           "fp4_quantize_noalloc")


def fp4_gemm_workspace_size(fmt: int, double_block: bool, M: int, N: int, K: int) -> int:
    n = _SZ(0)
    _check(_lib.fp4_gemm_workspace_size(fmt, int(double_block), M, N, K, ctypes.byref(n)), "fp4_gemm_workspace_size")
    return n.value


def fp4_gemm(fmt, double_block, a_codes, a_scales, a_outer, a_tensor_scale, b_codes, b_scales,
             b_outer, b_tensor_scale, M, N, K, c, out_dtype, ldc, workspace=None, workspace_bytes=0,
             stream=None) -> None:
    _check(_lib.fp4_gemm(fmt, int(double_block), _ptr(a_codes), _ptr(a_scales), _ptr(a_outer),
                         _ptr(a_tensor_scale), _ptr(b_codes), _ptr(b_scales), _ptr(b_outer),
                         _ptr(b_tensor_scale), M, N, K, _ptr(c), out_dtype, ldc, _ptr(workspace),
                         workspace_bytes, _stream(stream)),
           "fp4_gemm")


def fp4_last_error(stream=None) -> int:
    """Status of the device error word (FP4_OK or FP4_ERR_TIMEOUT); clears it."""
    return _lib.fp4_last_error(_stream(stream))


# --------------------------------------------------------------------------- helpers
# Device buffers for a quantized tensor, allocated with torch (plumbing only).

def in_dtype_of(x) -> int:
    import torch
    if x.dtype == torch.bfloat16:
        return FP4_IN_BF16
    if x.dtype == torch.float32:
        return FP4_IN_F32
    raise TypeError("input must be bfloat16 or float32, got %s" % x.dtype)


def alloc_qtensor(lines: int, K: int, fmt: int, double_block: bool = False, device="cuda"):
    """codes [L, K/2] u8, tiled scales, outer [L, K/128] f32 (double block), tensor scale f32."""
    import torch
    return dict(
        codes=torch.empty((lines, K // 2), dtype=torch.uint8, device=device),
        scales=torch.empty(max(fp4_scales_bytes(lines, K, fmt), 16), dtype=torch.uint8, device=device),
        outer=torch.empty((lines, max(K // 128, 1)), dtype=torch.float32, device=device) if double_block else None,
        tensor_scale=torch.empty(1, dtype=torch.float32, device=device),
        lines=lines, K=K, format=fmt, double_block=bool(double_block))


@_on_stream
def quantize(x, fmt, rounding=FP4_RTNE, rotation=FP4_ROT_NONE, axis=1, double_block=False, seed=0,
             tensor_id=0, tensor_amax=None, out=None, workspace=None, cols=None, stream=None):
    """Quantize a 2-D CUDA tensor (row-major, unit stride in the last dim) into a new or given qtensor."""
    import torch
    rows, ld = x.shape[0], x.stride(0) if x.dim() == 2 and x.shape[0] > 1 else x.shape[1]
    cols = x.shape[1] if cols is None else cols
    K, L = (cols, rows) if axis == 1 else (rows, cols)
    q = out if out is not None else alloc_qtensor(L, K, fmt, double_block, x.device)
    ws_bytes = fp4_quantize_workspace_size(fmt, double_block, tensor_amax is not None)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    fp4_quantize(x, in_dtype_of(x), rows, cols, ld, fmt, rounding, rotation, axis, double_block, seed,
                 tensor_id, tensor_amax, q["codes"], q["scales"], q["outer"], q["tensor_scale"],
                 workspace if ws_bytes else None, ws_bytes, stream)
    return q


def fp4_quantize_both_axes(x, in_dtype, rows, cols, ld, fmt, rotation, seed, rounding_rows, tensor_id_rows,
                           codes_rows, scales_rows, tensor_scale_rows, rounding_cols, tensor_id_cols, codes_cols,
                           scales_cols, tensor_scale_cols, workspace, workspace_bytes, stream=None) -> None:
    _check(_lib.fp4_quantize_both_axes(_ptr(x), in_dtype, rows, cols, ld, fmt, rotation, seed, rounding_rows,
                                       tensor_id_rows, _ptr(codes_rows), _ptr(scales_rows), _ptr(tensor_scale_rows),
                                       rounding_cols, tensor_id_cols, _ptr(codes_cols), _ptr(scales_cols),
                                       _ptr(tensor_scale_cols), _ptr(workspace), workspace_bytes, _stream(stream)),
           "fp4_quantize_both_axes")


@_on_stream
def quantize_both_axes(x, fmt, rotation=FP4_ROT_NONE, seed=0, rounding_rows=FP4_RTNE, tensor_id_rows=0,
                       rounding_cols=FP4_RTNE, tensor_id_cols=0, out_rows=None, out_cols=None, workspace=None,
                       stream=None):
    """Quantize a 2-D bf16 CUDA tensor along its rows and its columns in one pass;
    returns (qtensor of the rows, qtensor of the columns)."""
    import torch
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else cols
    qr = out_rows if out_rows is not None else alloc_qtensor(rows, cols, fmt, False, x.device)
    qc = out_cols if out_cols is not None else alloc_qtensor(cols, rows, fmt, False, x.device)
    if workspace is None:
        workspace = torch.empty(256, dtype=torch.uint8, device=x.device)
    fp4_quantize_both_axes(x, in_dtype_of(x), rows, cols, ld, fmt, rotation, seed, rounding_rows, tensor_id_rows,
                           qr["codes"], qr["scales"], qr["tensor_scale"], rounding_cols, tensor_id_cols,
                           qc["codes"], qc["scales"], qc["tensor_scale"], workspace, workspace.numel(), stream)
    return qr, qc


@_on_stream
def gemm(qa, qb, out_dtype=FP4_OUT_F32, out=None, workspace=None, stream=None):
    """C = A B^T on two quantized tensors of the same format (lines along K);
    UFP4 takes a workspace (allocated here when none is given)."""
    import torch
    M, N, K = qa["lines"], qb["lines"], qa["K"]
    if qb["K"] != K or qa["format"] != qb["format"] or qa["double_block"] != qb["double_block"]:
        raise ValueError("operands must share K, format and double-block mode")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16 if out_dtype == FP4_OUT_BF16 else torch.float32,
                          device=qa["codes"].device)
    ws_bytes = fp4_gemm_workspace_size(qa["format"], qa["double_block"], M, N, K)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=qa["codes"].device)
    fp4_gemm(qa["format"], qa["double_block"], qa["codes"], qa["scales"], qa["outer"], qa["tensor_scale"],
             qb["codes"], qb["scales"], qb["outer"], qb["tensor_scale"], M, N, K, out, out_dtype,
             out.stride(0), workspace if ws_bytes else None, ws_bytes, stream)
    return out


# --------------------------------------------------------------------------- OutControl

def fp4_channel_amax(x, in_dtype, rows, cols, ld, amax_out, stream=None) -> None:
    _check(_lib.fp4_channel_amax(_ptr(x), in_dtype, rows, cols, ld, _ptr(amax_out), _stream(stream)),
           "fp4_channel_amax")


def fp4_outctl_workspace_size(cols: int) -> int:
    n = _SZ(0)
    _check(_lib.fp4_outctl_workspace_size(cols, ctypes.byref(n)), "fp4_outctl_workspace_size")
    return n.value


def fp4_outctl_quantize(x, in_dtype, rows, cols, ld, channels, n_channels, k8, rounding, rotation, seed, tensor_id,
                        codes, scales, tensor_scale, codes8, scale8, workspace, workspace_bytes, stream=None) -> None:
    _check(_lib.fp4_outctl_quantize(_ptr(x), in_dtype, rows, cols, ld, _ptr(channels), n_channels, k8, rounding,
                                    rotation, seed, tensor_id, _ptr(codes), _ptr(scales), _ptr(tensor_scale),
                                    _ptr(codes8), _ptr(scale8), _ptr(workspace), workspace_bytes, _stream(stream)),
           "fp4_outctl_quantize")


def fp4_gemm_outctl(a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, a8_codes, a8_scale, b8_codes, b8_scale,
                    M, N, K, K8, c, out_dtype, ldc, stream=None) -> None:
    _check(_lib.fp4_gemm_outctl(_ptr(a_codes), _ptr(a_scales), _ptr(a_ts), _ptr(b_codes), _ptr(b_scales), _ptr(b_ts),
                                _ptr(a8_codes), _ptr(a8_scale), _ptr(b8_codes), _ptr(b8_scale), M, N, K, K8, _ptr(c),
                                out_dtype, ldc, _stream(stream)), "fp4_gemm_outctl")


@_on_stream
def channel_amax(x, stream=None):
    """max over rows of |x[:, c]| for a 2-D CUDA tensor (fp4_channel_amax)."""
    import torch
    rows, cols = x.shape
    out = torch.empty(max(cols, 1), dtype=torch.float32, device=x.device)
    fp4_channel_amax(x, in_dtype_of(x), rows, cols, x.stride(0) if rows > 1 else cols, out, stream)
    return out[:cols]


def outctl_channels(amax, p: float):
    """Calibration: the ceil(p * cols) channels with the largest amax (ties to
    the lower index), in ascending order, as a device int32 tensor."""
    import math
    import torch
    n = math.ceil(p * amax.numel())
    order = torch.sort(-amax, stable=True).indices[:n]
    return torch.sort(order).values.to(torch.int32)


@_on_stream
def outctl_quantize(x, channels, k8=None, rounding=FP4_RTNE, rotation=FP4_ROT_NONE, seed=0, tensor_id=0,
                    out=None, stream=None):
    """The OutControl split of a 2-D CUDA tensor along its channels
    (fp4_outctl_quantize): {"fp4": NVFP4 qtensor, "fp8": {"codes", "scale", "K"}}."""
    import torch
    rows, cols = x.shape
    n = channels.numel()
    k8 = (n + 127) // 128 * 128 if k8 is None else k8
    o = out if out is not None else dict(
        fp4=alloc_qtensor(rows, cols, FP4_NVFP4, False, x.device),
        fp8=dict(codes=torch.empty((rows, max(k8, 1)), dtype=torch.uint8, device=x.device),
                 scale=torch.empty(1, dtype=torch.float32, device=x.device), K=k8))
    ws = torch.empty(fp4_outctl_workspace_size(cols), dtype=torch.uint8, device=x.device)
    q4, q8 = o["fp4"], o["fp8"]
    fp4_outctl_quantize(x, in_dtype_of(x), rows, cols, x.stride(0) if rows > 1 else cols, channels, n, k8, rounding,
                        rotation, seed, tensor_id, q4["codes"], q4["scales"], q4["tensor_scale"], q8["codes"],
                        q8["scale"], ws, ws.numel(), stream)
    return o


@_on_stream
def gemm_outctl(qa, qb, out_dtype=FP4_OUT_F32, out=None, stream=None):
    """C = A B^T on two OutControl-split operands (fp4_gemm_outctl)."""
    import torch
    a4, b4, a8, b8 = qa["fp4"], qb["fp4"], qa["fp8"], qb["fp8"]
    M, N, K, K8 = a4["lines"], b4["lines"], a4["K"], a8["K"]
    if b4["K"] != K or b8["K"] != K8:
        raise ValueError("operands must share K and the FP8 width")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16 if out_dtype == FP4_OUT_BF16 else torch.float32,
                          device=a4["codes"].device)
    fp4_gemm_outctl(a4["codes"], a4["scales"], a4["tensor_scale"], b4["codes"], b4["scales"], b4["tensor_scale"],
                    a8["codes"], a8["scale"], b8["codes"], b8["scale"], M, N, K, K8, out, out_dtype, out.stride(0),
                    stream)
    return out


# --------------------------------------------------------------------------- FP8, a scale per block of 128

def fp4_fp8_block_scales_count(lines: int, K: int, block_lines: int) -> int:
    return _lib.fp4_fp8_block_scales_count(lines, K, block_lines)


def fp4_fp8_block_quantize(x, in_dtype, rows, cols, ld, block_lines, codes_rows, ld_rows, scales_rows, codes_cols,
                           ld_cols, scales_cols, stream=None) -> None:
    _check(_lib.fp4_fp8_block_quantize(_ptr(x), in_dtype, rows, cols, ld, block_lines, _ptr(codes_rows), ld_rows,
                                       _ptr(scales_rows), _ptr(codes_cols), ld_cols, _ptr(scales_cols),
                                       _stream(stream)), "fp4_fp8_block_quantize")


def fp4_fp8_block_gemm(a_codes, lda, a_scales, b_codes, ldb, b_scales, b_block_lines, M, N, K, c, out_dtype, ldc,
                       stream=None) -> None:
    _check(_lib.fp4_fp8_block_gemm(_ptr(a_codes), lda, _ptr(a_scales), _ptr(b_codes), ldb, _ptr(b_scales),
                                   b_block_lines, M, N, K, _ptr(c), out_dtype, ldc, _stream(stream)),
           "fp4_fp8_block_gemm")


# The helpers below look at every tensor before its address is handed on.  A call
# for one token takes a few microseconds on the GPU, so the checks read each
# property once and build their messages only when they fail.

def _device_of(t, what: str) -> int:
    """The device index of a CUDA tensor; the library launches on the current
    device, so a tensor of another one is refused."""
    import torch
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be a CUDA tensor" % what)
    if dev != torch.cuda.current_device():
        raise ValueError("%s is on %s, the current device is cuda:%d" % (what, t.device, torch.cuda.current_device()))
    return dev


def _mat(t, what: str, shape, dtype, dev) -> int:
    """Row pitch in elements of a [rows, cols] tensor with unit stride in its
    last dimension, of this type and on this device."""
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s is on %s, the other tensors on device %d" % (what, t.device, dev))
    ld, unit = t.stride()
    if unit != 1 and shape[1] > 1:
        raise ValueError("%s must have unit stride in its last dimension" % what)
    # the pitch of a single row is not used, and torch may call it anything
    return ld if shape[0] > 1 else (shape[1] + 15) // 16 * 16


def _flat(t, what: str, shape, dtype, dev):
    """A contiguous tensor of this shape and type on this device."""
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s is on %s, the other tensors on device %d" % (what, t.device, dev))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    return t


def alloc_fp8_block(lines: int, K: int, block_lines: int = 1, device="cuda"):
    """E4M3 codes [lines, K rounded up to 16] u8 and scales [ceil(K / 128), ...] f32 (include/fp4.h)."""
    import torch
    if block_lines not in (1, 128):
        raise ValueError("block_lines must be 1 or 128, got %r" % (block_lines,))
    n = (lines + 127) // 128 * (128 if block_lines == 1 else 1)
    return dict(codes=torch.empty((lines, (K + 15) // 16 * 16), dtype=torch.uint8, device=device),
                scales=torch.empty(((K + 127) // 128, n), dtype=torch.float32, device=device),
                lines=lines, K=K, block_lines=block_lines)


def _fp8_tensor(q, what: str, lines: int, K: int, block_lines: int, dev):
    """Address and pitch of the codes and address of the scales of an FP8 tensor, checked."""
    import torch
    codes, scales = q["codes"], q["scales"]
    if q["lines"] != lines or q["K"] != K or q["block_lines"] != block_lines or block_lines not in (1, 128):
        raise ValueError("%s must hold %d lines of %d in blocks of %d lines" % (what, lines, K, block_lines))
    width = codes.shape[-1]
    if width < K:
        raise ValueError("%s: codes must be [%d, >= %d], got %s" % (what, lines, K, tuple(codes.shape)))
    ld = _mat(codes, what + " codes", (lines, width), torch.uint8, dev)
    n = (lines + 127) // 128 * (128 if block_lines == 1 else 1)
    _flat(scales, what + " scales", ((K + 127) // 128, n), torch.float32, dev)
    return codes.data_ptr(), ld, scales.data_ptr()


_NO_FP8 = (None, 0, None)


def _fp8_quantize(x, block_lines, out_rows, out_cols, want_rows, want_cols, stream):
    dev = _device_of(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D, got %s" % (tuple(x.shape),))
    shape = rows, cols = x.shape
    dt, ld = in_dtype_of(x), _mat(x, "x", shape, x.dtype, dev)
    if want_rows and out_rows is None:
        out_rows = alloc_fp8_block(rows, cols, block_lines, x.device)
    if want_cols and out_cols is None:
        out_cols = alloc_fp8_block(cols, rows, block_lines, x.device)
    r = _fp8_tensor(out_rows, "the rows' result", rows, cols, block_lines, dev) if want_rows else _NO_FP8
    c = _fp8_tensor(out_cols, "the columns' result", cols, rows, block_lines, dev) if want_cols else _NO_FP8
    _check(_lib.fp4_fp8_block_quantize(x.data_ptr(), dt, rows, cols, ld, block_lines, *r, *c, _stream(stream)),
           "fp4_fp8_block_quantize")
    return out_rows, out_cols


@_on_stream
def fp8_block_quantize(x, axis=1, block_lines=1, out=None, stream=None):
    """E4M3 of a 2-D CUDA tensor with a scale per block of 128 along its rows
    (axis 1) or its columns (axis 0: the transposed tensor), of block_lines (1
    or 128) lines (fp4_fp8_block_quantize); into a new or given FP8 tensor
    {"codes", "scales", "lines", "K", "block_lines"}."""
    if axis == 1:
        return _fp8_quantize(x, block_lines, out, None, True, False, stream)[0]
    if axis == 0:
        return _fp8_quantize(x, block_lines, None, out, False, True, stream)[1]
    raise ValueError("axis must be 0 or 1, got %r" % (axis,))


@_on_stream
def fp8_block_quantize_both_axes(x, block_lines=1, out_rows=None, out_cols=None, stream=None):
    """fp8_block_quantize along the rows and along the columns from one read;
    returns (FP8 tensor of the rows, FP8 tensor of the columns)."""
    return _fp8_quantize(x, block_lines, out_rows, out_cols, True, True, stream)


@_on_stream
def fp8_block_gemm(qa, qb, out_dtype=FP4_OUT_F32, out=None, stream=None):
    """C = A B^T on two FP8 tensors (fp4_fp8_block_gemm): A in 1 x 128 blocks,
    B in 1 x 128 or 128 x 128 blocks."""
    import torch
    M, N, K = qa["lines"], qb["lines"], qa["K"]
    if qb["K"] != K or qa["block_lines"] != 1:
        raise ValueError("operands must share K, and A must have 1 x 128 blocks")
    dev = _device_of(qa["codes"], "A")
    a = _fp8_tensor(qa, "A", M, K, 1, dev)
    b = _fp8_tensor(qb, "B", N, K, qb["block_lines"], dev)
    dtype = torch.bfloat16 if out_dtype == FP4_OUT_BF16 else torch.float32
    if out is None:
        out = torch.empty((M, (N + 7) // 8 * 8), dtype=dtype, device=qa["codes"].device)[:, :N]
    ldc = _mat(out, "out", (M, N), dtype, dev)
    _check(_lib.fp4_fp8_block_gemm(*a, *b, qb["block_lines"], M, N, K, out.data_ptr(), out_dtype, ldc, _stream(stream)),
           "fp4_fp8_block_gemm")
    return out


# --------------------------------------------------------------------------- norms, gate and residual

def fp4_norm_residual(o, ldo, h, ldh, dtype, rows, cols, w_post, gate, ld_gate, rows_per_group, alpha, w_pre, eps,
                      h_out, ld_hout, y, ldy, codes, ld_codes, scales, rstd_post, rstd_pre, stream=None) -> None:
    _check(_lib.fp4_norm_residual(_ptr(o), ldo, _ptr(h), ldh, dtype, rows, cols, _ptr(w_post), _ptr(gate), ld_gate,
                                  rows_per_group, alpha, _ptr(w_pre), eps, _ptr(h_out), ld_hout, _ptr(y), ldy,
                                  _ptr(codes), ld_codes, _ptr(scales), _ptr(rstd_post), _ptr(rstd_pre),
                                  _stream(stream)), "fp4_norm_residual")


def fp4_norm_residual_backward_workspace_size(rows, cols, has_pre, has_post, has_gate, rows_per_group) -> int:
    n = _SZ(0)
    _check(_lib.fp4_norm_residual_backward_workspace_size(rows, cols, int(has_pre), int(has_post), int(has_gate),
                                                          rows_per_group, ctypes.byref(n)),
           "fp4_norm_residual_backward_workspace_size")
    return n.value


def fp4_norm_residual_backward(dy, lddy, dh_in, ld_dhin, h, ldh, o, ldo, dtype, rows, cols, w_post, gate, ld_gate,
                               rows_per_group, alpha, w_pre, rstd_post, rstd_pre, dh, ld_dh, d_o, ld_do, dw_pre,
                               dw_post, dgate, workspace, workspace_bytes, stream=None) -> None:
    _check(_lib.fp4_norm_residual_backward(_ptr(dy), lddy, _ptr(dh_in), ld_dhin, _ptr(h), ldh, _ptr(o), ldo, dtype,
                                           rows, cols, _ptr(w_post), _ptr(gate), ld_gate, rows_per_group, alpha,
                                           _ptr(w_pre), _ptr(rstd_post), _ptr(rstd_pre), _ptr(dh), ld_dh, _ptr(d_o),
                                           ld_do, _ptr(dw_pre), _ptr(dw_post), _ptr(dgate), _ptr(workspace),
                                           workspace_bytes, _stream(stream)), "fp4_norm_residual_backward")


def _opt_mat(t, what: str, shape, dtype, dev):
    """(address, row pitch) of an optional [rows, cols] tensor."""
    return (None, 0) if t is None else (t.data_ptr(), _mat(t, what, shape, dtype, dev))


def _opt_flat(t, what: str, shape, dtype, dev):
    """Address of an optional contiguous tensor."""
    return None if t is None else _flat(t, what, shape, dtype, dev).data_ptr()


def _gate_of(gate, rows_per_group, rows, cols, dtype, dev):
    """(address, row pitch, rows per group) of an optional gate."""
    if gate is None:
        return None, 0, 0
    if rows_per_group is None or rows_per_group < 1:
        raise ValueError("a gate needs rows_per_group >= 1")
    shape = ((rows + rows_per_group - 1) // rows_per_group, cols)
    # no more than the rows: the library's integers have 64 bits
    return gate.data_ptr(), _mat(gate, "gate", shape, dtype, dev), min(rows_per_group, max(rows, 1))


def _new_vector(t, what: str, shape, like, dev):
    """A given float32 buffer, checked, or a new one."""
    import torch
    if t is None:
        return torch.empty(shape, dtype=torch.float32, device=like.device)
    return _flat(t, what, shape, torch.float32, dev)


def _new_mat(t, like, shape):
    """A given buffer, or a new [rows, cols] tensor of like's type whose row pitch is a multiple of 16 bytes."""
    import torch
    if t is not None:
        return t
    return torch.empty((shape[0], (shape[1] + 7) // 8 * 8), dtype=like.dtype, device=like.device)[:, :shape[1]]


@_on_stream
def norm_residual(h, w_pre=None, o=None, w_post=None, gate=None, rows_per_group=None, alpha=1.0, eps=1e-6,
                  quantize=False, out=None, stream=None):
    """The norms after and before a block with its gate and the residual update
    (fp4_norm_residual) on 2-D CUDA tensors: h' = h + alpha * gate * (o, or its
    RMS norm times w_post), y = the RMS norm of h' times w_pre.  Returns {"h":
    h' (h itself without o), "rstd_post", "rstd_pre", and with w_pre "y", or
    with quantize=True "q", y as an FP8 tensor of 1 x 128 blocks}.  `out` may
    hold buffers under those names; out["y"] and out["q"] together get both."""
    out = out or {}
    if w_pre is None and (quantize or out.get("y") is not None or out.get("q") is not None):
        raise ValueError("y and q need the norm before the block: w_pre is not given")
    dev = _device_of(h, "h")
    if h.dim() != 2:
        raise ValueError("h must be 2-D, got %s" % (tuple(h.shape),))
    shape = rows, cols = h.shape
    dt, dtype = in_dtype_of(h), h.dtype
    ldh = _mat(h, "h", shape, dtype, dev)
    if o is None:
        if w_pre is None:
            raise ValueError("nothing to do: neither o nor w_pre is given")
        if w_post is not None or gate is not None:
            raise ValueError("w_post and gate belong to a block output o")
    got = dict(h=h, rstd_post=None, rstd_pre=None)
    po = ph = (None, 0)
    if o is not None:
        po = _opt_mat(o, "o", shape, dtype, dev)
        got["h"] = _new_mat(out.get("h"), h, shape)
        ph = _opt_mat(got["h"], "out h", shape, dtype, dev)
    p_post = _opt_flat(w_post, "w_post", (cols,), dtype, dev)
    p_pre = _opt_flat(w_pre, "w_pre", (cols,), dtype, dev)
    gate = _gate_of(gate, rows_per_group, rows, cols, dtype, dev)
    r_post = r_pre = None
    if w_post is not None:
        got["rstd_post"] = _new_vector(out.get("rstd_post"), "rstd_post", (rows,), h, dev)
        r_post = got["rstd_post"].data_ptr()
    y, q = (None, 0), _NO_FP8
    if w_pre is not None:
        got["rstd_pre"] = _new_vector(out.get("rstd_pre"), "rstd_pre", (rows,), h, dev)
        r_pre = got["rstd_pre"].data_ptr()
        given_y, given_q = out.get("y"), out.get("q")
        if quantize or given_q is not None:
            got["q"] = given_q if given_q is not None else alloc_fp8_block(rows, cols, 1, h.device)
            q = _fp8_tensor(got["q"], "q", rows, cols, 1, dev)
        if not quantize or given_y is not None:
            got["y"] = _new_mat(given_y, h, shape)
            y = _opt_mat(got["y"], "y", shape, dtype, dev)
    _check(_lib.fp4_norm_residual(*po, h.data_ptr(), ldh, dt, rows, cols, p_post, *gate, alpha, p_pre, eps, *ph, *y, *q,
                                  r_post, r_pre, _stream(stream)), "fp4_norm_residual")
    return got


@_on_stream
def norm_residual_backward(dy, h, rstd_pre=None, w_pre=None, dh_in=None, o=None, w_post=None, rstd_post=None,
                           gate=None, rows_per_group=None, alpha=1.0, out=None, workspace=None, stream=None):
    """The gradients of norm_residual (fp4_norm_residual_backward): dy of y, or
    None without a norm before the block; h the stream that norm_residual
    returned; dh_in the gradient that reaches it from elsewhere.  Returns
    {"dh", "do", "dw_pre", "dw_post", "dgate"}, None where it has no meaning;
    the last three in float32.  `out` may hold buffers under those names."""
    import torch
    like = dy if dy is not None else dh_in
    if like is None:
        raise ValueError("neither dy nor dh_in is given")
    dev = _device_of(like, "the incoming gradient")
    if like.dim() != 2:
        raise ValueError("the incoming gradient must be 2-D, got %s" % (tuple(like.shape),))
    shape = rows, cols = like.shape
    dt, dtype, f32, out = in_dtype_of(like), like.dtype, torch.float32, out or {}
    if (dy is None) != (w_pre is None) or (w_pre is not None and (rstd_pre is None or h is None)):
        raise ValueError("dy, w_pre, rstd_pre and h go together")
    if o is None and (w_post is not None or gate is not None):
        raise ValueError("w_post and gate belong to a block output o")
    if w_post is not None and rstd_post is None:
        raise ValueError("w_post and rstd_post go together")
    has_pre, has_post, has_gate = w_pre is not None, w_post is not None, gate is not None
    p_dy = _opt_mat(dy, "dy", shape, dtype, dev)
    p_in = _opt_mat(dh_in, "dh_in", shape, dtype, dev)
    p_h = _opt_mat(h if has_pre else None, "h", shape, dtype, dev)
    p_o = _opt_mat(o, "o", shape, dtype, dev)
    p_pre = _opt_flat(w_pre, "w_pre", (cols,), dtype, dev)
    p_post = _opt_flat(w_post, "w_post", (cols,), dtype, dev)
    r_pre = _opt_flat(rstd_pre if has_pre else None, "rstd_pre", (rows,), f32, dev)
    r_post = _opt_flat(rstd_post if has_post else None, "rstd_post", (rows,), f32, dev)
    gate_shape = gate.shape if has_gate else None
    gate = _gate_of(gate, rows_per_group, rows, cols, dtype, dev)
    got = dict(dh=_new_mat(out.get("dh"), like, shape), do=None, dw_pre=None, dw_post=None, dgate=None)
    p_dh, p_do, addr = _opt_mat(got["dh"], "out dh", shape, dtype, dev), (None, 0), [None, None, None]
    if o is not None:
        got["do"] = _new_mat(out.get("do"), like, shape)
        p_do = _opt_mat(got["do"], "out do", shape, dtype, dev)
    for i, (name, has, size) in enumerate((("dw_pre", has_pre, (cols,)), ("dw_post", has_post, (cols,)),
                                           ("dgate", has_gate, gate_shape))):
        if has:
            got[name] = _new_vector(out.get(name), name, size, like, dev)
            addr[i] = got[name].data_ptr()
    ws_bytes = fp4_norm_residual_backward_workspace_size(rows, cols, has_pre, has_post, has_gate, gate[2])
    ws = None
    if ws_bytes:
        if workspace is None:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=like.device)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous and on %s" % like.device)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(_lib.fp4_norm_residual_backward(*p_dy, *p_in, *p_h, *p_o, dt, rows, cols, p_post, *gate, alpha, p_pre, r_post,
                                           r_pre, *p_dh, *p_do, *addr, ws, ws_bytes, _stream(stream)),
           "fp4_norm_residual_backward")
    return got
