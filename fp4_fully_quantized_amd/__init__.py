"""Thin Python binding of libfp4.so (include/fp4.h), the gfx950 FP4 quantize +
FP4 GEMM library.

Argument marshalling only: every step of the path runs in the library's HIP
kernels. PyTorch supplies device memory and the stream. Importing this module
does not load the library; the first call does, and raises if it is missing
(build it with ``python -m fp4_fully_quantized_amd.build``).
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libfp4.so")

FP4_OK = 0
FP4_DTYPE_F32, FP4_DTYPE_BF16 = 0, 1
FP4_NVFP4, FP4_MXFP4 = 0, 1
FP4_RTN, FP4_SR = 0, 1
FP4_AXIS_COLS, FP4_AXIS_ROWS = 0, 1
FP4_OPERAND_QUANTIZED, FP4_OPERAND_RAW = 0, 1
FP4_LAYOUT_N, FP4_LAYOUT_T = 0, 1
FP4_ERR_WORKSPACE = 7
FP4_ACT_NONE, FP4_ACT_RELU, FP4_ACT_GELU, FP4_ACT_SILU = 0, 1, 2, 3
BLOCK = {FP4_NVFP4: 16, FP4_MXFP4: 32}

EXPORTS = ["fp4_codes_bytes", "fp4_scales_bytes", "fp4_hadamard_signs", "fp4_status_str",
           "fp4_tensor_amax", "fp4_tensor_amax_hadamard16", "fp4_quantize", "fp4_quantize_dual",
           "fp4_quantize_shard", "fp4_quantize_dual_shard", "fp4_quantize_noise", "fp4_quantize_dual_noise", "fp4_noise_ratio", "fp4_quantize_2d",
           "fp4_dequantize", "fp4_dequantize_unrotated", "fp4_gemm_workspace_bytes", "fp4_gemm_splitk_bytes", "fp4_gemm",
           "fp4_gemm_noalloc", "fp4_mx8_quantize", "fp4_mx8_dequantize", "fp4_rmsnorm", "fp4_rmsnorm_backward",
           "fp4_rmsnorm_backward_workspace_bytes", "fp4_gemm_fused", "fp4_gemm_fused_workspace_bytes",
           "fp4_act_backward", "fp4_act_backward_workspace_bytes"]
# The allocation-free GEMM's workspace limit (FP4_GEMM_NOALLOC_MAX_BYTES).
FP4_GEMM_NOALLOC_MAX_BYTES = 128 << 20


class Fp4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {fp4_status_str(status)} (status {status})")
        self.status = status


class fp4_tensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("amax", ctypes.c_void_p), ("tscale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("fmt", ctypes.c_int32), ("had_on", ctypes.c_int32),
                ("had_signs", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class fp4_operand(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("q", ctypes.POINTER(fp4_tensor)), ("data", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("k", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("layout", ctypes.c_int32), ("fmt", ctypes.c_int32), ("rnd", ctypes.c_int32),
                ("had_on", ctypes.c_int32), ("seed", ctypes.c_uint64), ("index_offset", ctypes.c_uint64),
                ("had_signs", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class fp4_mx8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("ld", ctypes.c_int64), ("lds", ctypes.c_int64)]


class fp4_rmsnorm_fwd(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("gamma_t", ctypes.c_int32), ("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64),
                ("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64), ("gamma", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("ld_h", ctypes.c_int64), ("y", ctypes.c_void_p), ("ld_y", ctypes.c_int64),
                ("y8", ctypes.POINTER(fp4_mx8)), ("h8", ctypes.POINTER(fp4_mx8)), ("rstd", ctypes.c_void_p),
                ("amax", ctypes.c_void_p), ("eps", ctypes.c_float), ("reserved", ctypes.c_uint32)]


class fp4_rmsnorm_bwd(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("gamma_t", ctypes.c_int32), ("dy", ctypes.c_void_p), ("ld_dy", ctypes.c_int64),
                ("h", ctypes.c_void_p), ("ld_h", ctypes.c_int64), ("h8", ctypes.POINTER(fp4_mx8)),
                ("gamma", ctypes.c_void_p), ("rstd", ctypes.c_void_p), ("dres", ctypes.c_void_p),
                ("ld_dres", ctypes.c_int64), ("dx", ctypes.c_void_p), ("ld_dx", ctypes.c_int64),
                ("dgamma", ctypes.c_void_p), ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t)]


class fp4_epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64),
                ("z8", ctypes.POINTER(fp4_mx8)), ("bias_t", ctypes.c_int32), ("residual_t", ctypes.c_int32),
                ("act", ctypes.c_int32), ("reserved", ctypes.c_uint32)]


class fp4_act_bwd(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("act", ctypes.c_int32), ("dy", ctypes.c_void_p), ("ld_dy", ctypes.c_int64), ("z", ctypes.c_void_p),
                ("ld_z", ctypes.c_int64), ("z8", ctypes.POINTER(fp4_mx8)), ("dz", ctypes.c_void_p),
                ("ld_dz", ctypes.c_int64), ("dbias", ctypes.c_void_p), ("amax", ctypes.c_void_p),
                ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t)]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run python -m fp4_fully_quantized_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        c = ctypes
        L.fp4_codes_bytes.restype = c.c_size_t
        L.fp4_codes_bytes.argtypes = [c.c_int64, c.c_int64]
        L.fp4_scales_bytes.restype = c.c_size_t
        L.fp4_scales_bytes.argtypes = [c.c_int64, c.c_int64, c.c_int32]
        L.fp4_hadamard_signs.restype = c.c_uint32
        L.fp4_hadamard_signs.argtypes = [c.c_uint64]
        L.fp4_status_str.restype = c.c_char_p
        L.fp4_status_str.argtypes = [c.c_int]
        L.fp4_tensor_amax.restype = c.c_int
        L.fp4_tensor_amax.argtypes = [c.c_void_p, c.c_int, c.c_int64, c.c_int64, c.c_int64,
                                      c.c_void_p, c.c_void_p]
        L.fp4_tensor_amax_hadamard16.restype = c.c_int
        L.fp4_tensor_amax_hadamard16.argtypes = [c.c_void_p, c.c_int, c.c_int64, c.c_int64, c.c_int64,
                                                 c.c_int, c.c_uint32, c.c_void_p, c.c_void_p]
        L.fp4_quantize.restype = c.c_int
        L.fp4_quantize.argtypes = [c.c_void_p, c.c_int, c.c_int64, c.c_int64, c.c_int64, c.c_int,
                                   c.c_int, c.c_uint64, c.c_uint64, c.c_int,
                                   c.POINTER(fp4_tensor), c.c_void_p]
        L.fp4_quantize_dual.restype = c.c_int
        L.fp4_quantize_dual.argtypes = [c.c_void_p, c.c_int, c.c_int64, c.c_int64, c.c_int64,
                                        c.c_int, c.c_uint64, c.c_uint64, c.c_int, c.c_uint64, c.c_uint64,
                                        c.c_int, c.POINTER(fp4_tensor), c.POINTER(fp4_tensor), c.c_void_p]
        L.fp4_quantize_shard.restype = c.c_int
        L.fp4_quantize_shard.argtypes = (L.fp4_quantize.argtypes[:5] + [c.c_int64, c.c_int64]
                                         + L.fp4_quantize.argtypes[5:-1] + [c.c_void_p, c.c_void_p])
        L.fp4_quantize_dual_shard.restype = c.c_int
        L.fp4_quantize_dual_shard.argtypes = (L.fp4_quantize_dual.argtypes[:5] + [c.c_int64, c.c_int64]
                                              + L.fp4_quantize_dual.argtypes[5:-1]
                                              + [c.c_void_p, c.c_void_p, c.c_void_p])
        L.fp4_quantize_noise.restype = c.c_int
        L.fp4_quantize_noise.argtypes = L.fp4_quantize.argtypes[:-1] + [c.c_void_p, c.c_void_p]
        L.fp4_quantize_dual_noise.restype = c.c_int
        L.fp4_quantize_dual_noise.argtypes = L.fp4_quantize_dual.argtypes[:-1] + [c.c_void_p, c.c_void_p,
                                                                                  c.c_void_p]
        L.fp4_quantize_2d.restype = c.c_int
        L.fp4_quantize_2d.argtypes = [c.c_void_p, c.c_int, c.c_int64, c.c_int64, c.c_int64, c.c_int,
                                      c.c_uint64, c.c_uint64, c.c_int, c.POINTER(fp4_tensor),
                                      c.POINTER(fp4_tensor), c.c_void_p]
        L.fp4_dequantize.restype = c.c_int
        L.fp4_dequantize_unrotated.restype = c.c_int
        L.fp4_dequantize_unrotated.argtypes = [c.POINTER(fp4_tensor), c.c_int, c.c_void_p, c.c_int64,
                                               c.c_void_p]
        L.fp4_dequantize.argtypes = [c.POINTER(fp4_tensor), c.c_int, c.c_void_p, c.c_int64,
                                     c.c_void_p]
        L.fp4_noise_ratio.restype = c.c_int
        L.fp4_noise_ratio.argtypes = [c.c_void_p, c.c_void_p, c.c_void_p]
        L.fp4_gemm_workspace_bytes.restype = c.c_size_t
        L.fp4_gemm_workspace_bytes.argtypes = [c.POINTER(fp4_operand), c.POINTER(fp4_operand)]
        L.fp4_gemm_splitk_bytes.restype = c.c_size_t
        L.fp4_gemm_splitk_bytes.argtypes = [c.POINTER(fp4_operand), c.POINTER(fp4_operand)]
        L.fp4_gemm.restype = c.c_int
        L.fp4_gemm.argtypes = [c.POINTER(fp4_operand), c.POINTER(fp4_operand), c.c_int, c.c_void_p,
                               c.c_int64, c.c_void_p, c.c_size_t, c.c_void_p]
        L.fp4_gemm_noalloc.restype = c.c_int
        L.fp4_gemm_noalloc.argtypes = [c.POINTER(fp4_operand), c.POINTER(fp4_operand), c.c_int, c.c_void_p,
                                       c.c_int64, c.c_void_p]
        L.fp4_mx8_quantize.restype = c.c_int
        L.fp4_mx8_quantize.argtypes = [c.c_void_p, c.c_int, c.c_int64, c.POINTER(fp4_mx8), c.c_void_p]
        L.fp4_mx8_dequantize.restype = c.c_int
        L.fp4_mx8_dequantize.argtypes = [c.POINTER(fp4_mx8), c.c_int, c.c_void_p, c.c_int64, c.c_void_p]
        L.fp4_rmsnorm.restype = c.c_int
        L.fp4_rmsnorm.argtypes = [c.POINTER(fp4_rmsnorm_fwd), c.c_void_p]
        L.fp4_rmsnorm_backward.restype = c.c_int
        L.fp4_rmsnorm_backward.argtypes = [c.POINTER(fp4_rmsnorm_bwd), c.c_void_p]
        L.fp4_rmsnorm_backward_workspace_bytes.restype = c.c_size_t
        L.fp4_rmsnorm_backward_workspace_bytes.argtypes = [c.c_int64, c.c_int64]
        L.fp4_gemm_fused.restype = c.c_int
        L.fp4_gemm_fused.argtypes = [c.POINTER(fp4_operand), c.POINTER(fp4_operand), c.POINTER(fp4_epilogue),
                                     c.c_int, c.c_void_p, c.c_int64, c.c_void_p, c.c_size_t, c.c_void_p]
        L.fp4_gemm_fused_workspace_bytes.restype = c.c_size_t
        L.fp4_gemm_fused_workspace_bytes.argtypes = [c.POINTER(fp4_operand), c.POINTER(fp4_operand)]
        L.fp4_act_backward.restype = c.c_int
        L.fp4_act_backward.argtypes = [c.POINTER(fp4_act_bwd), c.c_void_p]
        L.fp4_act_backward_workspace_bytes.restype = c.c_size_t
        L.fp4_act_backward_workspace_bytes.argtypes = [c.c_int64, c.c_int64]
        _lib = L
    return _lib


# ---------------------------------------------------------------- raw ABI calls
def fp4_codes_bytes(rows: int, cols: int) -> int:
    return lib().fp4_codes_bytes(rows, cols)


def fp4_scales_bytes(rows: int, cols: int, fmt: int) -> int:
    return lib().fp4_scales_bytes(rows, cols, fmt)


def fp4_hadamard_signs(seed: int) -> int:
    return lib().fp4_hadamard_signs(seed)


def fp4_status_str(status: int) -> str:
    return lib().fp4_status_str(status).decode()


def _check(status: int, what: str) -> None:
    if status != FP4_OK:
        raise Fp4Error(status, what)


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return FP4_DTYPE_BF16
    if t.dtype == torch.float32:
        return FP4_DTYPE_F32
    raise TypeError(f"FP4 library takes float32 or bfloat16 tensors, got {t.dtype}")


# ---------------------------------------------------------------- argument checks
# The library checks shapes, alignment and enums, but it sees raw pointers: it
# cannot tell a host pointer, a tensor that is too small or a transposed view
# from a good one. These checks run before every call that passes tensors.
def _check_device(t, name: str, device=None):
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a tensor on a GPU (got device {getattr(t, 'device', None)})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other arguments on {device}")


def _check_matrix(t, name: str, device=None):
    """A 2-D float32/bfloat16 device matrix, row-major with unit column stride."""
    _check_device(t, name, device)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    _dtype_code(t)
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must be row-major with unit column stride")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} rows overlap (stride {t.stride(0)} < {t.shape[1]} columns)")


def _check_scalar(t, name: str, dtype, count: int, device):
    import torch
    _check_device(t, name, device)
    if t.dtype != dtype or t.numel() < count or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} device tensor of at least {count} element(s)")
    del torch


def _check_qtensor(q, name: str, device=None, amax: bool = False):
    """The QTensor's buffers exist on the device and hold rows x cols codes and
    scales; amax: the call needs the tensor amax too (NVFP4)."""
    import torch
    if not isinstance(q, QTensor):
        raise TypeError(f"{name} must be a QTensor")
    device = device or q.codes.device
    for part, t, need in (("codes", q.codes, fp4_codes_bytes(q.rows, q.cols)),
                          ("scales", q.scales, fp4_scales_bytes(q.rows, q.cols, q.fmt))):
        _check_device(t, f"{name}.{part}", device)
        if t.dtype != torch.uint8 or not t.is_contiguous():
            raise ValueError(f"{name}.{part} must be a contiguous uint8 tensor")
        if need == 0 or t.numel() < need:
            raise ValueError(f"{name}.{part} holds {t.numel()} bytes, {q.rows} x {q.cols} needs {need}")
    if q.fmt == FP4_NVFP4:
        if amax or q.amax is not None:
            _check_scalar(q.amax, f"{name}.amax", torch.float32, 1, device)
            if amax and q.tscale is not None and q.amax.data_ptr() == q.tscale.data_ptr():
                raise ValueError(f"{name}.amax and {name}.tscale are one tensor")
        _check_scalar(q.tscale, f"{name}.tscale", torch.float32, 1, device)


def _check_quant_out(src, out, axis: int, name: str = "out"):
    """The output QTensor has the quantized orientation of src."""
    R, C = src.shape
    want = (C, R) if axis == FP4_AXIS_ROWS else (R, C)
    if (out.rows, out.cols) != want:
        raise ValueError(f"{name} is {out.rows} x {out.cols}; quantizing a {R} x {C} source along "
                         f"{'rows' if axis == FP4_AXIS_ROWS else 'cols'} needs {want[0]} x {want[1]}")
    _check_qtensor(out, name, src.device, amax=True)


def _amax_of(x):
    """The tensor amax of amax_from: of a QTensor, or of a result that has one."""
    if getattr(x, "amax", None) is None:
        raise ValueError("amax_from has no amax")
    return x.amax


# ---------------------------------------------------------------- tensors
class QTensor:
    """A quantized matrix (quantized orientation rows x cols) held in torch
    device tensors, and its fp4_tensor descriptor."""

    def __init__(self, rows: int, cols: int, fmt: int, device="cuda", had_signs: int | None = None):
        import torch
        B = BLOCK[fmt]
        if cols % B:
            raise ValueError(f"cols={cols} is not a multiple of the block size {B}")
        self.rows, self.cols, self.fmt = rows, cols, fmt
        self.codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=device)
        self.scales = torch.empty((rows, cols // B), dtype=torch.uint8, device=device)
        if fmt == FP4_NVFP4:
            self.amax = torch.zeros(1, dtype=torch.float32, device=device)
            self.tscale = torch.zeros(1, dtype=torch.float32, device=device)
        else:
            self.amax = self.tscale = None
        self.had_on = had_signs is not None
        self.had_signs = int(had_signs or 0)

    @classmethod
    def wrap(cls, codes, scales, fmt: int, amax=None, tscale=None, had_signs: int | None = None) -> "QTensor":
        """A QTensor on tensors the caller has (a loaded weight, a slice of
        whole rows): codes uint8 [rows, cols / 2], scales uint8 [rows, cols / B],
        both contiguous; NVFP4 needs tscale. Products and dequantizations need
        no amax; without one the tensor serves neither as a quantization's
        output nor as amax_from. Checked by the calls that take it."""
        q = cls.__new__(cls)
        q.rows, q.cols, q.fmt = codes.shape[0], 2 * codes.shape[1], fmt
        q.codes, q.scales = codes, scales
        q.tscale = tscale if fmt == FP4_NVFP4 else None
        q.amax = amax if fmt == FP4_NVFP4 else None
        q.had_on = had_signs is not None
        q.had_signs = int(had_signs or 0)
        return q

    def desc(self) -> fp4_tensor:
        d = fp4_tensor()
        d.codes = self.codes.data_ptr()
        d.scales = self.scales.data_ptr()
        d.amax = self.amax.data_ptr() if self.amax is not None else None
        d.tscale = self.tscale.data_ptr() if self.tscale is not None else None
        d.rows, d.cols = self.rows, self.cols
        d.fmt = self.fmt
        d.had_on = int(self.had_on)
        d.had_signs = self.had_signs
        return d


def fp4_tensor_amax(src, amax, stream=None) -> None:
    import torch
    _check_matrix(src, "src")
    _check_scalar(amax, "amax", torch.float32, 1, src.device)
    R, C = src.shape
    _check(lib().fp4_tensor_amax(src.data_ptr(), _dtype_code(src), R, C, src.stride(0),
                                 amax.data_ptr(), _stream(stream)), "fp4_tensor_amax")


def fp4_tensor_amax_hadamard16(src, axis: int, had_signs: int, amax, stream=None) -> None:
    import torch
    _check_matrix(src, "src")
    _check_scalar(amax, "amax", torch.float32, 1, src.device)
    R, C = src.shape
    _check(lib().fp4_tensor_amax_hadamard16(src.data_ptr(), _dtype_code(src), R, C, src.stride(0),
                                            axis, had_signs, amax.data_ptr(), _stream(stream)),
           "fp4_tensor_amax_hadamard16")


def fp4_quantize(src, axis: int, rnd: int, seed: int, index_offset: int, amax_ready: bool,
                 out: QTensor, stream=None) -> None:
    _check_matrix(src, "src")
    _check_quant_out(src, out, axis)
    R, C = src.shape
    d = out.desc()
    _check(lib().fp4_quantize(src.data_ptr(), _dtype_code(src), R, C, src.stride(0), axis, rnd,
                              seed, index_offset, int(bool(amax_ready)), ctypes.byref(d),
                              _stream(stream)), "fp4_quantize")
    out.rows, out.cols = d.rows, d.cols


def fp4_quantize_dual(src, rnd_cols: int, seed_cols: int, index_offset_cols: int, rnd_rows: int,
                      seed_rows: int, index_offset_rows: int, amax_ready: bool, out_cols: QTensor,
                      out_rows: QTensor, stream=None) -> None:
    _check_matrix(src, "src")
    _check_quant_out(src, out_cols, FP4_AXIS_COLS, "out_cols")
    _check_quant_out(src, out_rows, FP4_AXIS_ROWS, "out_rows")
    R, C = src.shape
    dc, dr = out_cols.desc(), out_rows.desc()
    _check(lib().fp4_quantize_dual(src.data_ptr(), _dtype_code(src), R, C, src.stride(0), rnd_cols,
                                   seed_cols, index_offset_cols, rnd_rows, seed_rows, index_offset_rows,
                                   int(bool(amax_ready)), ctypes.byref(dc), ctypes.byref(dr),
                                   _stream(stream)), "fp4_quantize_dual")
    out_cols.rows, out_cols.cols = dc.rows, dc.cols
    out_rows.rows, out_rows.cols = dr.rows, dr.cols


def fp4_quantize_shard(src, row_offset: int, rows_total: int, axis: int, rnd: int, seed: int,
                       index_offset: int, amax_ready: bool, out: QTensor, noise=None, stream=None) -> None:
    """fp4_quantize of rows row_offset .. of a rows_total-row tensor, with the
    whole tensor's stochastic-rounding indices (noise: None, or the float64
    device tensor of 2 sums of fp4_quantize_noise)."""
    import torch
    _check_matrix(src, "src")
    _check_quant_out(src, out, axis)
    if noise is not None:
        _check_scalar(noise, "noise", torch.float64, 2, src.device)
    R, C = src.shape
    d = out.desc()
    _check(lib().fp4_quantize_shard(src.data_ptr(), _dtype_code(src), R, C, src.stride(0), row_offset,
                                    rows_total, axis, rnd, seed, index_offset, int(bool(amax_ready)),
                                    ctypes.byref(d), _ptr(noise), _stream(stream)), "fp4_quantize_shard")
    out.rows, out.cols = d.rows, d.cols


def fp4_quantize_dual_shard(src, row_offset: int, rows_total: int, rnd_cols: int, seed_cols: int,
                            index_offset_cols: int, rnd_rows: int, seed_rows: int, index_offset_rows: int,
                            amax_ready: bool, out_cols: QTensor, out_rows: QTensor, noise_cols=None,
                            noise_rows=None, stream=None) -> None:
    """fp4_quantize_dual of a row shard, with the whole tensor's stochastic-rounding indices."""
    import torch
    _check_matrix(src, "src")
    _check_quant_out(src, out_cols, FP4_AXIS_COLS, "out_cols")
    _check_quant_out(src, out_rows, FP4_AXIS_ROWS, "out_rows")
    for nm, t in (("noise_cols", noise_cols), ("noise_rows", noise_rows)):
        if t is not None:
            _check_scalar(t, nm, torch.float64, 2, src.device)
    R, C = src.shape
    dc, dr = out_cols.desc(), out_rows.desc()
    _check(lib().fp4_quantize_dual_shard(src.data_ptr(), _dtype_code(src), R, C, src.stride(0), row_offset,
                                         rows_total, rnd_cols, seed_cols, index_offset_cols, rnd_rows,
                                         seed_rows, index_offset_rows, int(bool(amax_ready)), ctypes.byref(dc),
                                         ctypes.byref(dr), _ptr(noise_cols), _ptr(noise_rows), _stream(stream)),
           "fp4_quantize_dual_shard")
    out_cols.rows, out_cols.cols = dc.rows, dc.cols
    out_rows.rows, out_rows.cols = dr.rows, dr.cols


def _ptr(t):
    return None if t is None else t.data_ptr()


def fp4_quantize_noise(src, axis: int, rnd: int, seed: int, index_offset: int, amax_ready: bool,
                       out: QTensor, noise, stream=None) -> None:
    """fp4_quantize plus noise[0] += sum x^2, noise[1] += sum (xhat - x)^2
    (noise: a float64 device tensor of 2 elements)."""
    import torch
    _check_matrix(src, "src")
    _check_quant_out(src, out, axis)
    _check_scalar(noise, "noise", torch.float64, 2, src.device)
    R, C = src.shape
    d = out.desc()
    _check(lib().fp4_quantize_noise(src.data_ptr(), _dtype_code(src), R, C, src.stride(0), axis, rnd,
                                    seed, index_offset, int(bool(amax_ready)), ctypes.byref(d),
                                    _ptr(noise), _stream(stream)), "fp4_quantize_noise")
    out.rows, out.cols = d.rows, d.cols


def fp4_quantize_dual_noise(src, rnd_cols: int, seed_cols: int, index_offset_cols: int, rnd_rows: int,
                            seed_rows: int, index_offset_rows: int, amax_ready: bool, out_cols: QTensor,
                            out_rows: QTensor, noise_cols=None, noise_rows=None, stream=None) -> None:
    import torch
    _check_matrix(src, "src")
    _check_quant_out(src, out_cols, FP4_AXIS_COLS, "out_cols")
    _check_quant_out(src, out_rows, FP4_AXIS_ROWS, "out_rows")
    for nm, t in (("noise_cols", noise_cols), ("noise_rows", noise_rows)):
        if t is not None:
            _check_scalar(t, nm, torch.float64, 2, src.device)
    R, C = src.shape
    dc, dr = out_cols.desc(), out_rows.desc()
    _check(lib().fp4_quantize_dual_noise(src.data_ptr(), _dtype_code(src), R, C, src.stride(0),
                                         rnd_cols, seed_cols, index_offset_cols, rnd_rows, seed_rows,
                                         index_offset_rows, int(bool(amax_ready)), ctypes.byref(dc),
                                         ctypes.byref(dr), _ptr(noise_cols), _ptr(noise_rows),
                                         _stream(stream)), "fp4_quantize_dual_noise")
    out_cols.rows, out_cols.cols = dc.rows, dc.cols
    out_rows.rows, out_rows.cols = dr.rows, dr.cols


def fp4_quantize_2d(src, rnd: int, seed: int, index_offset: int, amax_ready: bool, out: QTensor,
                    out_t: QTensor, stream=None) -> None:
    _check_matrix(src, "src")
    _check_quant_out(src, out, FP4_AXIS_COLS, "out")
    _check_quant_out(src, out_t, FP4_AXIS_ROWS, "out_t")
    R, C = src.shape
    d, dt = out.desc(), out_t.desc()
    _check(lib().fp4_quantize_2d(src.data_ptr(), _dtype_code(src), R, C, src.stride(0), rnd, seed,
                                 index_offset, int(bool(amax_ready)), ctypes.byref(d), ctypes.byref(dt),
                                 _stream(stream)), "fp4_quantize_2d")
    out.rows, out.cols = d.rows, d.cols
    out_t.rows, out_t.cols = dt.rows, dt.cols


def quantize_2d(src, fmt: int = FP4_NVFP4, rnd: int = FP4_RTN, seed: int = 0, index_offset: int = 0,
                amax_from: QTensor | None = None, stream=None):
    """Allocate both QTensors and quantize src with B x B blocks. Returns
    (q [R, C] blocked along C, q_t [C, R] blocked along R), one quantization
    sharing the tensor amax (NVFP4)."""
    R, C = src.shape
    q = QTensor(R, C, fmt, device=src.device)
    qt = QTensor(C, R, fmt, device=src.device)
    ready = False
    if amax_from is not None and fmt == FP4_NVFP4:
        q.amax = _amax_of(amax_from)
        ready = True
    if fmt == FP4_NVFP4:
        qt.amax = q.amax
    fp4_quantize_2d(src, rnd, seed, index_offset, ready, q, qt, stream)
    return q, qt


def fp4_noise_ratio(noise, ratio, stream=None) -> None:
    """ratio[0] = sqrt(noise[0] / noise[1]), computed by the library on the
    device in stream order (noise: 2 float64, ratio: 1 float64, device)."""
    import torch
    _check_scalar(noise, "noise", torch.float64, 2, None)
    _check_scalar(ratio, "ratio", torch.float64, 1, noise.device)
    _check(lib().fp4_noise_ratio(noise.data_ptr(), ratio.data_ptr(), _stream(stream)), "fp4_noise_ratio")


def noise_ratio(noise, stream=None):
    """The monitor's ratio ||g|| / ||Q(g) - g|| as a 1-element float64 device
    tensor (fp4_noise_ratio into a new tensor)."""
    import torch
    ratio = torch.empty(1, dtype=torch.float64, device=noise.device)
    fp4_noise_ratio(noise, ratio, stream)
    return ratio


def fp4_dequantize(q: QTensor, dst, stream=None) -> None:
    _dequantize("fp4_dequantize", q, dst, stream)


def fp4_dequantize_unrotated(q: QTensor, dst, stream=None) -> None:
    """fp4_dequantize, then the inverse of the quantization's block rotation
    (when q.had_on): the values in the tensor's own domain."""
    _dequantize("fp4_dequantize_unrotated", q, dst, stream)


def _dequantize(name, q, dst, stream):
    _check_qtensor(q, "q")
    _check_matrix(dst, "dst", q.codes.device)
    if tuple(dst.shape) != (q.rows, q.cols):
        raise ValueError(f"dst is {tuple(dst.shape)}, q is {q.rows} x {q.cols}")
    d = q.desc()
    _check(getattr(lib(), name)(ctypes.byref(d), _dtype_code(dst), dst.data_ptr(), dst.stride(0),
                                _stream(stream)), name)


class RawOperand:
    """A GEMM operand that fp4_gemm quantizes into its workspace first: the
    rows x K matrix `data` (layout N: data is rows x K) or its transpose
    (layout T: data is K x rows), with the format, rounding, SR stream and
    rotation of fp4_quantize."""

    def __init__(self, data, layout: int = FP4_LAYOUT_N, fmt: int = FP4_NVFP4, rnd: int = FP4_RTN,
                 seed: int = 0, index_offset: int = 0, had_signs: int | None = None):
        _check_matrix(data, "data")
        if layout not in (FP4_LAYOUT_N, FP4_LAYOUT_T):
            raise ValueError(f"layout must be FP4_LAYOUT_N or FP4_LAYOUT_T, got {layout}")
        self.data, self.layout, self.fmt, self.rnd = data, layout, fmt, rnd
        self.seed, self.index_offset = seed, index_offset
        self.had_on = had_signs is not None
        self.had_signs = int(had_signs or 0)
        R, C = data.shape
        self.rows, self.k = (C, R) if layout == FP4_LAYOUT_T else (R, C)

    @property
    def device(self):
        return self.data.device

    def operand(self) -> fp4_operand:
        o = fp4_operand()
        o.kind = FP4_OPERAND_RAW
        o.dtype = _dtype_code(self.data)
        o.data = self.data.data_ptr()
        o.rows, o.k, o.ld = self.rows, self.k, self.data.stride(0)
        o.layout, o.fmt, o.rnd = self.layout, self.fmt, self.rnd
        o.had_on, o.had_signs = int(self.had_on), self.had_signs
        o.seed, o.index_offset = self.seed, self.index_offset
        return o


def _operand(x, name: str):
    """(fp4_operand, keep-alive) for a QTensor or a RawOperand."""
    if isinstance(x, RawOperand):
        return x.operand(), None
    _check_qtensor(x, name)
    d = x.desc()
    o = fp4_operand()
    o.kind = FP4_OPERAND_QUANTIZED
    o.q = ctypes.pointer(d)
    return o, d


def _operand_device(x):
    return x.device if isinstance(x, RawOperand) else x.codes.device


def fp4_gemm_workspace_bytes(A, B) -> int:
    oa, ka = _operand(A, "A")
    ob, kb = _operand(B, "B")
    return lib().fp4_gemm_workspace_bytes(ctypes.byref(oa), ctypes.byref(ob))


def fp4_gemm_splitk_bytes(A, B) -> int:
    oa, ka = _operand(A, "A")
    ob, kb = _operand(B, "B")
    return lib().fp4_gemm_splitk_bytes(ctypes.byref(oa), ctypes.byref(ob))


def fp4_gemm(A, B, C, ws=None, stream=None) -> None:
    """C = A_hat B_hat^T (FP32 accumulation). A and B are QTensors blocked
    along K or RawOperands (quantized into `ws`, a uint8 device tensor of at
    least fp4_gemm_workspace_bytes(A, B) bytes; with fp4_gemm_splitk_bytes(A, B)
    more, the last partial wave of output tiles is split along K)."""
    import torch
    dev = _operand_device(A)
    if _operand_device(B) != dev:
        raise ValueError(f"A is on {dev}, B on {_operand_device(B)}")
    oa, ka = _operand(A, "A")
    ob, kb = _operand(B, "B")
    _check_matrix(C, "C", dev)
    if tuple(C.shape) != (A.rows, B.rows):
        raise ValueError(f"C is {tuple(C.shape)}, the product is {A.rows} x {B.rows}")
    ws_ptr, ws_bytes = None, 0
    if ws is not None:
        _check_device(ws, "ws", dev)
        if ws.dtype != torch.uint8 or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous uint8 device tensor")
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel()
    _check(lib().fp4_gemm(ctypes.byref(oa), ctypes.byref(ob), _dtype_code(C), C.data_ptr(), C.stride(0),
                          ws_ptr, ws_bytes, _stream(stream)), "fp4_gemm")


def fp4_gemm_noalloc(A, B, C, stream=None) -> None:
    """fp4_gemm with the library's own static workspace (for callers that
    cannot allocate): RAW operands are quantized there. Calls with RAW
    operands that overlap on one GPU race on that workspace."""
    dev = _operand_device(A)
    if _operand_device(B) != dev:
        raise ValueError(f"A is on {dev}, B on {_operand_device(B)}")
    oa, ka = _operand(A, "A")
    ob, kb = _operand(B, "B")
    _check_matrix(C, "C", dev)
    if tuple(C.shape) != (A.rows, B.rows):
        raise ValueError(f"C is {tuple(C.shape)}, the product is {A.rows} x {B.rows}")
    _check(lib().fp4_gemm_noalloc(ctypes.byref(oa), ctypes.byref(ob), _dtype_code(C), C.data_ptr(),
                                  C.stride(0), _stream(stream)), "fp4_gemm_noalloc")


# ---------------------------------------------------------------- conveniences
def quantize(src, axis: int = FP4_AXIS_COLS, fmt: int = FP4_NVFP4, rnd: int = FP4_RTN,
             seed: int = 0, index_offset: int = 0, had_signs: int | None = None,
             amax_from: QTensor | None = None, noise=None, stream=None) -> QTensor:
    """Allocate a QTensor and quantize src into it. `amax_from`: reuse the
    tensor amax already computed for the same tensor (NVFP4). `noise`: a float64
    device tensor of 2 elements that the quantization noise sums are added to."""
    R, C = src.shape
    rows, cols = (C, R) if axis == FP4_AXIS_ROWS else (R, C)
    q = QTensor(rows, cols, fmt, device=src.device, had_signs=had_signs)
    ready = False
    if amax_from is not None and fmt == FP4_NVFP4:
        q.amax = _amax_of(amax_from)
        ready = True
    if noise is None:
        fp4_quantize(src, axis, rnd, seed, index_offset, ready, q, stream)
    else:
        fp4_quantize_noise(src, axis, rnd, seed, index_offset, ready, q, noise, stream)
    return q


def quantize_dual(src, fmt: int = FP4_NVFP4, rnd_cols: int = FP4_RTN, seed_cols: int = 0,
                  index_offset_cols: int = 0, rnd_rows: int = FP4_SR, seed_rows: int = 0,
                  index_offset_rows: int = 0, had_signs_cols: int | None = None,
                  had_signs_rows: int | None = None, amax_from: QTensor | None = None,
                  noise_cols=None, noise_rows=None, stream=None):
    """Allocate both QTensors and quantize src along C and along R in one
    read. Returns (q_cols [R, C], q_rows [C, R]). NVFP4 without rotation: they
    share the tensor amax (`amax_from`: a QTensor whose amax to reuse). NVFP4
    with a rotation on either side: each keeps its own amax (`amax_from`: a
    pair of QTensors, for the cols and the rows orientation)."""
    R, C = src.shape
    qc = QTensor(R, C, fmt, device=src.device, had_signs=had_signs_cols)
    qr = QTensor(C, R, fmt, device=src.device, had_signs=had_signs_rows)
    ready = False
    two = fmt == FP4_NVFP4 and (qc.had_on or qr.had_on)
    if amax_from is not None and fmt == FP4_NVFP4:
        if two:
            qc.amax, qr.amax = _amax_of(amax_from[0]), _amax_of(amax_from[1])
        else:
            qc.amax = _amax_of(amax_from)
        ready = True
    if fmt == FP4_NVFP4 and not two:
        qr.amax = qc.amax
    if noise_cols is None and noise_rows is None:
        fp4_quantize_dual(src, rnd_cols, seed_cols, index_offset_cols, rnd_rows, seed_rows,
                          index_offset_rows, ready, qc, qr, stream)
    else:
        fp4_quantize_dual_noise(src, rnd_cols, seed_cols, index_offset_cols, rnd_rows, seed_rows,
                                index_offset_rows, ready, qc, qr, noise_cols, noise_rows, stream)
    return qc, qr


def dequantize(q: QTensor, dtype=None, stream=None, unrotate=False):
    """Allocate the output and run fp4_dequantize (fp4_dequantize_unrotated
    with unrotate=True)."""
    import torch
    dst = torch.empty((q.rows, q.cols), dtype=dtype or torch.float32, device=q.codes.device)
    (fp4_dequantize_unrotated if unrotate else fp4_dequantize)(q, dst, stream)
    return dst


def gemm(A, B, dtype=None, out=None, ws=None, stream=None):
    """Allocate the output (and, when none is given, the workspace: the RAW
    operands' and the split-K area) and run fp4_gemm."""
    import torch
    dev = _operand_device(A)
    if out is None:
        out = torch.empty((A.rows, B.rows), dtype=dtype or torch.float32, device=dev)
    if ws is None:
        n = fp4_gemm_workspace_bytes(A, B) + fp4_gemm_splitk_bytes(A, B)
        if n:
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
    fp4_gemm(A, B, out, ws, stream)
    return out


# ---------------------------------------------------------------- around the product
# These calls also run once per token of a serving loop, where the host's own
# time shows: arguments are looked at once, a good one on a short path, and only
# a bad one goes through the checks above, which say what is wrong with it.
def _raw_stream(stream, device):
    import torch
    if stream is not None:
        return stream.cuda_stream
    return torch.cuda.current_stream(device).cuda_stream


def _fast_raw_stream():
    # The handle alone, without a Stream object around it (0.1 us for 2.8).
    import torch
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if get is None:
        return _raw_stream

    def raw(stream, device):
        return stream.cuda_stream if stream is not None else get(device.index)
    return raw


def _raw(stream, device):
    """The stream's handle for a call on device, which must be the current one (a launch goes there)."""
    global _raw
    import torch
    fast, current = _fast_raw_stream(), torch.cuda.current_device

    def raw(stream, device):
        if current() != device.index:
            raise ValueError(f"the tensors are on {device}, the current device is cuda:{current()}")
        return fast(stream, device)
    _raw = raw
    return raw(stream, device)


def _mat(t, name: str, device, shape=None, dtype=None) -> int:
    """Leading dimension of a 2-D float32/bfloat16 device matrix with unit
    column stride and rows that do not overlap (ValueError / TypeError)."""
    if not (getattr(t, "is_cuda", False) and (device is None or t.device == device)):
        _check_device(t, name, device)
    size = t.shape
    if shape is not None and size != shape:
        raise ValueError(f"{name} is {tuple(size)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if len(size) == 2:
        rows, cols = size
        ld, step = t.stride()
        if rows == 1:
            ld = max(cols, 1)   # whatever torch left there
        if (step == 1 or cols == 1) and ld >= cols:
            return ld
    _check_matrix(t, name, device)
    return max(size[1], 1)      # an empty matrix: the library refuses its shape


def _vec(t, name: str, n: int, device, dtype=None) -> int:
    """Data pointer of a vector of n values on device."""
    if not (getattr(t, "is_cuda", False) and t.device == device):
        _check_device(t, name, device)
    if dtype is None:
        _dtype_code(t)
    elif t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n} values, got shape {tuple(t.shape)}")
    return t.data_ptr()


def _new(shape, dtype, device, stream):
    """A tensor of the stream the call runs on, so that torch's allocator hands
    its memory out again only behind that stream's work. Strides are named: a
    norm of one token, three tensors, takes 13.5 us a call against 14.5 (calls with
    one output the same within 0.2 us)."""
    import torch
    if stream is None:
        return torch.empty_strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class MX8Tensor:
    """A rows x cols matrix in 8 bits (E4M3 values, one E8M0 scale byte per 32
    values of a row): codes uint8 [rows, ld] with ld = cols up to a multiple of
    32, scales uint8 [rows, ceil(cols / 32)]."""

    def __init__(self, rows: int, cols: int, device="cuda", stream=None):
        import torch
        blocks = (cols + 31) // 32
        self.rows, self.cols = rows, cols
        self.codes = _new((rows, 32 * blocks), torch.uint8, device, stream)
        self.scales = _new((rows, blocks), torch.uint8, device, stream)

    @classmethod
    def wrap(cls, codes, scales, cols: int) -> "MX8Tensor":
        """An MX8Tensor on tensors the caller has (unit column strides, whole blocks in each row of
        codes). Checked by the calls that take it."""
        q = cls.__new__(cls)
        q.rows, q.cols, q.codes, q.scales = codes.shape[0], cols, codes, scales
        return q

    def e4m3(self):
        """The codes as E4M3 values [rows, cols] (a view; each counts its block's scale)."""
        import torch
        return self.codes.view(torch.float8_e4m3fn)[:, :self.cols]

    def e8m0(self):
        """The scales as powers of two [rows, ceil(cols / 32)] (a view)."""
        import torch
        return self.scales.view(torch.float8_e8m0fnu)

    def desc(self) -> fp4_mx8:
        return _mx8(self, "tensor", None)


def _mx8(q, name: str, device, shape=None) -> fp4_mx8:
    """The descriptor of an MX8Tensor whose buffers hold what it says."""
    import torch
    if not isinstance(q, MX8Tensor):
        raise TypeError(f"{name} must be an MX8Tensor")
    rows, cols = q.rows, q.cols
    if shape is not None and (rows, cols) != tuple(shape):
        raise ValueError(f"{name} is {rows} x {cols}, expected {shape[0]} x {shape[1]}")
    blocks = (cols + 31) // 32
    codes, scales = q.codes, q.scales
    _check_device(codes, f"{name}.codes", device)
    _check_device(scales, f"{name}.scales", codes.device)
    for part, t, width in (("codes", codes, 32 * blocks), ("scales", scales, blocks)):
        if t.dtype != torch.uint8 or t.dim() != 2 or t.shape[0] != rows or t.shape[1] < width:
            raise ValueError(f"{name}.{part} must be uint8 [{rows}, {width}], got {t.dtype} {tuple(t.shape)}")
        if (t.shape[1] > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < width):
            raise ValueError(f"{name}.{part} must be row-major with unit column stride")
    # A single row's stride is whatever torch left there.
    ld, lds = (codes.stride(0), scales.stride(0)) if rows > 1 else (32 * blocks, blocks)
    return fp4_mx8(codes.data_ptr(), scales.data_ptr(), rows, cols, ld, lds)


def fp4_mx8_quantize(src, out: MX8Tensor, stream=None) -> None:
    ld = _mat(src, "src", None)
    _mx8_quantize(src, ld, _mx8(out, "out", src.device, src.shape), stream)


def _mx8_quantize(src, ld, d, stream):
    _check(lib().fp4_mx8_quantize(src.data_ptr(), _dtype_code(src), ld, ctypes.byref(d), _raw(stream, src.device)),
           "fp4_mx8_quantize")


def fp4_mx8_dequantize(q: MX8Tensor, dst, stream=None) -> None:
    d = _mx8(q, "q", None)
    _mx8_dequantize(d, dst, _mat(dst, "dst", q.codes.device, (q.rows, q.cols)), stream)


def _mx8_dequantize(d, dst, ld, stream):
    _check(lib().fp4_mx8_dequantize(ctypes.byref(d), _dtype_code(dst), dst.data_ptr(), ld, _raw(stream, dst.device)),
           "fp4_mx8_dequantize")


def mx8_quantize(src, stream=None) -> MX8Tensor:
    """src in 8 bits (a new MX8Tensor)."""
    ld = _mat(src, "src", None)
    q = MX8Tensor(src.shape[0], src.shape[1], src.device, stream)
    _mx8_quantize(src, ld, _own_mx8(q), stream)
    return q


def mx8_dequantize(q: MX8Tensor, dtype=None, stream=None):
    """The matrix q stands for (float32 unless dtype says otherwise)."""
    import torch
    d = _mx8(q, "q", None)
    dst = _new((q.rows, q.cols), dtype or torch.float32, q.codes.device, stream)
    _mx8_dequantize(d, dst, q.cols, stream)
    return dst


def _own_mx8(q) -> fp4_mx8:
    """The descriptor of an MX8Tensor made here."""
    blocks = (q.cols + 31) // 32
    return fp4_mx8(q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols, 32 * blocks, blocks)


def fp4_rmsnorm(x, gamma, eps: float, residual=None, h=None, y=None, y8=None, h8=None, rstd=None, amax=None,
                stream=None) -> None:
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * gamma into the outputs
    that are given (h, y like x; y8, h8 MX8Tensors; rstd float32 [rows]; amax a
    float32 scalar, max |y|)."""
    import torch
    n = _rmsnorm_in(x, gamma, eps, residual)
    dev, shape = x.device, x.shape
    if h is not None:
        n.ld_h, n.h = _mat(h, "h", dev, shape, x.dtype), h.data_ptr()
    if y is not None:
        n.ld_y, n.y = _mat(y, "y", dev, shape, x.dtype), y.data_ptr()
    if y8 is not None:
        n.y8 = ctypes.pointer(_mx8(y8, "y8", dev, shape))
    if h8 is not None:
        n.h8 = ctypes.pointer(_mx8(h8, "h8", dev, shape))
    if rstd is not None:
        n.rstd = _vec(rstd, "rstd", shape[0], dev, torch.float32)
    if amax is not None:
        _check_scalar(amax, "amax", torch.float32, 1, dev)
        n.amax = amax.data_ptr()
    _check(lib().fp4_rmsnorm(ctypes.byref(n), _raw(stream, dev)), "fp4_rmsnorm")


def _rmsnorm_in(x, gamma, eps, residual) -> fp4_rmsnorm_fwd:
    """The call's inputs, checked."""
    ld = _mat(x, "x", None)
    dev, shape = x.device, x.shape
    n = fp4_rmsnorm_fwd(shape[0], shape[1], _dtype_code(x), _dtype_code(gamma), x.data_ptr(), ld)
    n.gamma, n.eps = _vec(gamma, "gamma", shape[1], dev), eps
    if residual is not None:
        n.ld_residual, n.residual = _mat(residual, "residual", dev, shape, x.dtype), residual.data_ptr()
    return n


class RMSNorm(NamedTuple):
    """What rmsnorm computed: h (x itself without a residual), y, y8, h8, rstd,
    amax; None where it was not asked for. With amax it serves as quantize's
    amax_from for y."""
    h: object
    y: object
    y8: object
    h8: object
    rstd: object
    amax: object


def rmsnorm(x, gamma, eps: float = 1e-5, residual=None, y: bool = True, y8: bool = False, h8: bool = False,
            amax: bool = False, stream=None) -> RMSNorm:
    """Allocate the outputs and run fp4_rmsnorm. y8: y in 8 bits; h8: the
    checkpoint rmsnorm_backward reads; amax: max |y| (NVFP4's quantization
    of y then needs no pass of its own for it)."""
    import torch
    n = _rmsnorm_in(x, gamma, eps, residual)
    (rows, cols), dev = x.shape, x.device
    hm, ym, y8t, h8t, top = x, None, None, None, None
    rstd = _new((rows,), torch.float32, dev, stream)
    n.rstd = rstd.data_ptr()
    if residual is not None:
        hm = _new((rows, cols), x.dtype, dev, stream)
        n.h, n.ld_h = hm.data_ptr(), cols
    if y:
        ym = _new((rows, cols), x.dtype, dev, stream)
        n.y, n.ld_y = ym.data_ptr(), cols
    if y8:
        y8t = MX8Tensor(rows, cols, dev, stream)
        n.y8 = ctypes.pointer(_own_mx8(y8t))
    if h8:
        h8t = MX8Tensor(rows, cols, dev, stream)
        n.h8 = ctypes.pointer(_own_mx8(h8t))
    if amax:
        top = _new((1,), torch.float32, dev, stream)
        n.amax = top.data_ptr()
    _check(lib().fp4_rmsnorm(ctypes.byref(n), _raw(stream, dev)), "fp4_rmsnorm")
    return RMSNorm(hm, ym, y8t, h8t, rstd, top)


def fp4_rmsnorm_backward_workspace_bytes(rows: int, cols: int) -> int:
    return lib().fp4_rmsnorm_backward_workspace_bytes(rows, cols)


def _ws(ws, device):
    """(pointer, bytes) of a caller's workspace."""
    import torch
    if ws is None:
        return None, 0
    _check_device(ws, "ws", device)
    if ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 device tensor")
    return ws.data_ptr(), ws.numel()


def _rmsnorm_bwd_in(dy, h, gamma, rstd, dres) -> fp4_rmsnorm_bwd:
    """The call's inputs, checked."""
    import torch
    ld = _mat(dy, "dy", None)
    dev, shape = dy.device, dy.shape
    n = fp4_rmsnorm_bwd(shape[0], shape[1], _dtype_code(dy), _dtype_code(gamma), dy.data_ptr(), ld)
    n.gamma = _vec(gamma, "gamma", shape[1], dev)
    n.rstd = _vec(rstd, "rstd", shape[0], dev, torch.float32)
    if isinstance(h, MX8Tensor):
        n.h8 = ctypes.pointer(_mx8(h, "h", dev, shape))
    else:
        n.ld_h, n.h = _mat(h, "h", dev, shape, dy.dtype), h.data_ptr()
    if dres is not None:
        n.ld_dres, n.dres = _mat(dres, "dres", dev, shape, dy.dtype), dres.data_ptr()
    return n


def fp4_rmsnorm_backward(dy, h, gamma, rstd, dx, dgamma=None, dres=None, ws=None, stream=None) -> None:
    """dx = rstd (dy gamma - xhat mean(dy gamma xhat)) + dres and dgamma = sum
    dy xhat with xhat = h rstd; h a matrix or its MX8Tensor."""
    import torch
    n = _rmsnorm_bwd_in(dy, h, gamma, rstd, dres)
    n.ld_dx, n.dx = _mat(dx, "dx", dy.device, dy.shape, dy.dtype), dx.data_ptr()
    if dgamma is not None:
        n.dgamma = _vec(dgamma, "dgamma", dy.shape[1], dy.device, torch.float32)
    n.ws, n.ws_bytes = _ws(ws, dy.device)
    _check(lib().fp4_rmsnorm_backward(ctypes.byref(n), _raw(stream, dy.device)), "fp4_rmsnorm_backward")


def rmsnorm_backward(dy, h, gamma, rstd, dres=None, stream=None):
    """Allocate dx (like dy), dgamma (float32) and the workspace and run
    fp4_rmsnorm_backward. Returns (dx, dgamma)."""
    import torch
    n = _rmsnorm_bwd_in(dy, h, gamma, rstd, dres)
    (rows, cols), dev = dy.shape, dy.device
    dx = _new((rows, cols), dy.dtype, dev, stream)
    dgamma = _new((cols,), torch.float32, dev, stream)
    n.dx, n.ld_dx, n.dgamma = dx.data_ptr(), cols, dgamma.data_ptr()
    need = fp4_rmsnorm_backward_workspace_bytes(rows, cols)
    if need:
        ws = _new((need,), torch.uint8, dev, stream)
        n.ws, n.ws_bytes = ws.data_ptr(), need
    _check(lib().fp4_rmsnorm_backward(ctypes.byref(n), _raw(stream, dev)), "fp4_rmsnorm_backward")
    return dx, dgamma


def _product(x, name: str):
    """(fp4_operand, keep-alive) of a product's operand, as _operand."""
    import torch
    if not isinstance(x, QTensor):
        return _operand(x, name)
    c, s = x.codes, x.scales
    rows, cols, fmt = x.rows, x.cols, x.fmt
    nv = fmt == FP4_NVFP4
    if not (c.is_cuda and c.device == s.device and c.dtype == s.dtype == torch.uint8 and c.is_contiguous()
            and s.is_contiguous() and rows > 0 and cols > 0 and cols % BLOCK[fmt] == 0 and c.numel() >= rows * cols // 2
            and s.numel() >= rows * cols // BLOCK[fmt]
            and (not nv or (getattr(x.tscale, "dtype", None) == torch.float32 and x.tscale.device == c.device))):
        _check_qtensor(x, name)
    d = fp4_tensor(c.data_ptr(), s.data_ptr(), None, x.tscale.data_ptr() if nv else None, rows, cols, fmt, int(x.had_on),
                   x.had_signs)   # a product reads no amax
    return fp4_operand(FP4_OPERAND_QUANTIZED, 0, ctypes.pointer(d)), d


def fp4_gemm_fused_workspace_bytes(A, B) -> int:
    oa, ka = _operand(A, "A")
    ob, kb = _operand(B, "B")
    return lib().fp4_gemm_fused_workspace_bytes(ctypes.byref(oa), ctypes.byref(ob))


def _same_device(A, B):
    dev = _operand_device(A)
    if _operand_device(B) != dev:
        raise ValueError(f"A is on {dev}, B on {_operand_device(B)}")
    return dev


def _epilogue(dev, shape, bias, act, residual) -> fp4_epilogue:
    """The epilogue's inputs, checked."""
    e = fp4_epilogue()
    e.act = act
    if bias is not None:
        e.bias, e.bias_t = _vec(bias, "bias", shape[1], dev), _dtype_code(bias)
    if residual is not None:
        e.ld_residual, e.residual = _mat(residual, "residual", dev, shape), residual.data_ptr()
        e.residual_t = _dtype_code(residual)
    return e


def fp4_gemm_fused(A, B, C, bias=None, act: int = FP4_ACT_NONE, residual=None, z8=None, ws=None, stream=None) -> None:
    """C = act(A_hat B_hat^T + bias) + residual; z8: an MX8Tensor that receives
    the pre-activation. ws: at least fp4_gemm_workspace_bytes(A, B) bytes, or
    fp4_gemm_fused_workspace_bytes(A, B) to allow splitting along K."""
    dev = _same_device(A, B)
    oa, ka = _product(A, "A")
    ob, kb = _product(B, "B")
    shape = (A.rows, B.rows)
    e = _epilogue(dev, shape, bias, act, residual)
    ldc = _mat(C, "C", dev, shape)
    if z8 is not None:
        e.z8 = ctypes.pointer(_mx8(z8, "z8", dev, shape))
    ws_ptr, ws_bytes = _ws(ws, dev)
    _check(lib().fp4_gemm_fused(ctypes.byref(oa), ctypes.byref(ob), ctypes.byref(e), _dtype_code(C), C.data_ptr(), ldc,
                                ws_ptr, ws_bytes, _raw(stream, dev)), "fp4_gemm_fused")


def gemm_fused(A, B, bias=None, act: int = FP4_ACT_NONE, residual=None, checkpoint: bool = False, dtype=None,
               out=None, ws=None, stream=None):
    """Allocate the output, the pre-activation's 8-bit checkpoint (when asked
    for) and the workspace (when none is given) and run fp4_gemm_fused. Returns
    (out, z8), z8 None without checkpoint."""
    import torch
    dev = _same_device(A, B)
    oa, ka = _product(A, "A")
    ob, kb = _product(B, "B")
    a, b = ctypes.byref(oa), ctypes.byref(ob)
    shape = (A.rows, B.rows)
    e = _epilogue(dev, shape, bias, act, residual)
    if out is None:
        out = _new(shape, dtype or torch.float32, dev, stream)
        ldc = shape[1]
    else:
        ldc = _mat(out, "out", dev, shape)
    z8 = None
    if checkpoint:
        z8 = MX8Tensor(shape[0], shape[1], dev, stream)
        e.z8 = ctypes.pointer(_own_mx8(z8))
    if ws is None:
        n = lib().fp4_gemm_fused_workspace_bytes(a, b)
        if n:
            ws = _new((n,), torch.uint8, dev, stream)
    ws_ptr, ws_bytes = _ws(ws, dev)
    _check(lib().fp4_gemm_fused(a, b, ctypes.byref(e), _dtype_code(out), out.data_ptr(), ldc, ws_ptr, ws_bytes,
                                _raw(stream, dev)), "fp4_gemm_fused")
    return out, z8


class ActGrad(NamedTuple):
    """What act_backward computed; with amax it serves as quantize's amax_from for dz."""
    dz: object
    dbias: object
    amax: object


def fp4_act_backward_workspace_bytes(rows: int, cols: int) -> int:
    return lib().fp4_act_backward_workspace_bytes(rows, cols)


def _act_bwd_in(dy, z, act) -> fp4_act_bwd:
    """The call's inputs, checked."""
    ld = _mat(dy, "dy", None)
    dev, shape = dy.device, dy.shape
    n = fp4_act_bwd(shape[0], shape[1], _dtype_code(dy), act, dy.data_ptr(), ld)
    if isinstance(z, MX8Tensor):
        n.z8 = ctypes.pointer(_mx8(z, "z", dev, shape))
    else:
        n.ld_z, n.z = _mat(z, "z", dev, shape, dy.dtype), z.data_ptr()
    return n


def fp4_act_backward(dy, z, act: int, dz, dbias=None, amax=None, ws=None, stream=None) -> None:
    """dz = dy act'(z), dbias = sum over rows of dz, amax = max |dz|; z a matrix
    or the MX8Tensor that fp4_gemm_fused left."""
    import torch
    n = _act_bwd_in(dy, z, act)
    dev = dy.device
    n.ld_dz, n.dz = _mat(dz, "dz", dev, dy.shape, dy.dtype), dz.data_ptr()
    if dbias is not None:
        n.dbias = _vec(dbias, "dbias", dy.shape[1], dev, torch.float32)
    if amax is not None:
        _check_scalar(amax, "amax", torch.float32, 1, dev)
        n.amax = amax.data_ptr()
    n.ws, n.ws_bytes = _ws(ws, dev)
    _check(lib().fp4_act_backward(ctypes.byref(n), _raw(stream, dev)), "fp4_act_backward")


def act_backward(dy, z, act: int, dbias: bool = True, amax: bool = False, stream=None) -> ActGrad:
    """Allocate dz (like dy), dbias, amax and the workspace and run
    fp4_act_backward; None where not asked for."""
    import torch
    n = _act_bwd_in(dy, z, act)
    (rows, cols), dev = dy.shape, dy.device
    dz = _new((rows, cols), dy.dtype, dev, stream)
    n.dz, n.ld_dz = dz.data_ptr(), cols
    db = top = None
    if dbias:
        db = _new((cols,), torch.float32, dev, stream)
        n.dbias = db.data_ptr()
    if amax:
        top = _new((1,), torch.float32, dev, stream)
        n.amax = top.data_ptr()
    need = fp4_act_backward_workspace_bytes(rows, cols) if dbias or amax else 0
    if need:
        ws = _new((need,), torch.uint8, dev, stream)
        n.ws, n.ws_bytes = ws.data_ptr(), need
    _check(lib().fp4_act_backward(ctypes.byref(n), _raw(stream, dev)), "fp4_act_backward")
    return ActGrad(dz, db, top)
