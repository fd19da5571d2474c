"""Row-scaled NVFP4 quantize-transpose for AMD Instinct MI355X (gfx950).

A thin ctypes binding over ``libnvfp4.so`` (the C ABI declared in
``include/nvfp4.h``). Every function here has the name of the C entry point
it calls and only marshals arguments: it checks dtypes, shapes, contiguity
and devices of torch tensors, passes their device pointers and the current
HIP stream, and raises on a non-zero status. All computation runs in the HIP
kernels; there is no CPU fallback, and importing a function whose library is
missing raises.

Layouts (row-major, packed, no pitch):
  x      [M, K] bfloat16 or float32
  q_row  [M, ceil(K/2)] uint8   s_row [M, ceil(K/16)] uint8 (or float8_e4m3fn)
  q_col  [K, ceil(M/2)] uint8   s_col [K, ceil(M/16)] uint8 (or float8_e4m3fn)
"""
from __future__ import annotations

import ctypes
import importlib
import os
from typing import Optional

import torch

from .build import calls_path, library_path

NVFP4_OK = 0
NVFP4_ERR_ARG = -1
NVFP4_ERR_UNSUPPORTED = -2
NVFP4_ERR_HIP = -3

NVFP4_BF16 = 0
NVFP4_FP32 = 1

NVFP4_AMAX_TENSOR = 0
NVFP4_AMAX_LINE = 1
NVFP4_AMAX_ROWGROUP = 2

NVFP4_FLAG_FORCE_TWO_KERNEL = 1

NVFP4_FMT_NONE = 0
NVFP4_FMT_E4M3 = 1
NVFP4_FMT_NVFP4 = 2
NVFP4_FMT_INT8 = 3

NVFP4_ACT_NONE = 0
NVFP4_ACT_GELU = 1
NVFP4_ACT_SILU = 2
NVFP4_ACT_RELU2 = 3
NVFP4_ACT_SWIGLU = 4

# Every entry point include/nvfp4.h declares.
EXPORTED = ("nvfp4_amax_path", "nvfp4_amax_rowcol", "nvfp4_group_amax_expand",
            "nvfp4_check_group_end",
            "nvfp4_quantize_transpose", "nvfp4_quantize_rowcol", "nvfp4_quantize_4over6",
            "nvfp4_quantize_2d",
            "nvfp4_quantize_grouped",
            "nvfp4_quantize_dequantize", "nvfp4_dequantize",
            "nvfp4_gemm",
            "nvfp4_act_backward", "nvfp4_act_backward_workspace",
            "nvfp4_rmsnorm", "nvfp4_rmsnorm_backward", "nvfp4_rmsnorm_backward_workspace",
            "nvfp4_int8_quantize", "nvfp4_int8_quantize_rowcol", "nvfp4_int8_gemm",
            "nvfp4_layernorm", "nvfp4_layernorm_backward", "nvfp4_layernorm_backward_workspace",
            "nvfp4_cache_write", "nvfp4_cache_read",
            "nvfp4_status_string")

NVFP4_GROUPS_MAX = 256

_lib = None


class Nvfp4Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


def load_library():
    """Load libnvfp4.so (built in-tree by __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with __graft_entry__.build() "
                          "(the HIP library is required; there is no fallback)")
    lib = ctypes.CDLL(path)
    vp, f32p, u8p, i64p = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
    i64, c_int, c_uint, c_f = ctypes.c_int64, ctypes.c_int, ctypes.c_uint, ctypes.c_float
    lib.nvfp4_status_string.restype = ctypes.c_char_p
    lib.nvfp4_status_string.argtypes = [c_int]
    lib.nvfp4_amax_path.restype = c_int
    lib.nvfp4_amax_path.argtypes = [c_int, i64, i64, c_int, c_int, c_uint]
    lib.nvfp4_amax_rowcol.restype = c_int
    lib.nvfp4_amax_rowcol.argtypes = [vp, c_int, i64, i64, f32p, f32p, f32p, f32p, c_uint, vp]
    lib.nvfp4_group_amax_expand.restype = c_int
    lib.nvfp4_group_amax_expand.argtypes = [f32p, i64, i64p, i64, vp, f32p, vp]
    lib.nvfp4_check_group_end.restype = c_int
    lib.nvfp4_check_group_end.argtypes = [i64p, i64, i64]
    lib.nvfp4_quantize_transpose.restype = c_int
    lib.nvfp4_quantize_transpose.argtypes = [vp, c_int, i64, i64, c_int, f32p, c_int, f32p, c_f,
                                             u8p, u8p, u8p, u8p, f32p, vp]
    lib.nvfp4_quantize_4over6.restype = c_int
    lib.nvfp4_quantize_rowcol.restype = c_int
    lib.nvfp4_quantize_rowcol.argtypes = [vp, c_int, i64, i64, c_f, f32p, f32p, u8p, u8p, u8p, u8p,
                                          f32p, vp]
    lib.nvfp4_quantize_4over6.argtypes = [vp, c_int, i64, i64, c_int, f32p, c_int, f32p, c_f,
                                          u8p, u8p, u8p, u8p, f32p, vp]
    lib.nvfp4_quantize_2d.restype = c_int
    lib.nvfp4_quantize_2d.argtypes = [vp, c_int, i64, i64, f32p, c_f, u8p, u8p, u8p, u8p, f32p, vp]
    lib.nvfp4_quantize_grouped.restype = c_int
    lib.nvfp4_quantize_grouped.argtypes = [vp, c_int, i64, i64, i64p, i64, i64, i64, c_f, f32p,
                                           u8p, u8p, u8p, u8p, f32p, vp]
    lib.nvfp4_quantize_dequantize.restype = c_int
    lib.nvfp4_quantize_dequantize.argtypes = [vp, c_int, i64, i64, c_int, f32p, c_f, u8p, u8p, vp,
                                              c_int, f32p, vp]
    lib.nvfp4_dequantize.restype = c_int
    lib.nvfp4_dequantize.argtypes = [u8p, u8p, i64, i64, c_int, f32p, c_f, vp, c_int, f32p, vp]
    lib.nvfp4_gemm.restype = c_int
    lib.nvfp4_gemm.argtypes = [c_int, u8p, u8p, c_int, f32p, c_f, u8p, u8p, c_int, f32p, c_f,
                               i64, i64, i64, vp, c_int, c_int, vp, vp, vp, c_int, f32p, vp]
    lib.nvfp4_act_backward.restype = c_int
    lib.nvfp4_act_backward.argtypes = [vp, vp, c_int, i64, i64, c_int, vp, f32p, vp, i64, f32p, vp]
    lib.nvfp4_act_backward_workspace.restype = i64
    lib.nvfp4_act_backward_workspace.argtypes = [i64, i64, c_int]
    lib.nvfp4_rmsnorm.restype = c_int
    lib.nvfp4_rmsnorm.argtypes = [vp, vp, c_int, vp, c_int, c_f, i64, i64, vp, vp, c_int, f32p, c_int,
                                  u8p, u8p, f32p, c_f, f32p, vp]
    lib.nvfp4_rmsnorm_backward.restype = c_int
    lib.nvfp4_rmsnorm_backward.argtypes = [vp, vp, c_int, vp, c_int, f32p, vp, i64, i64, vp, f32p, vp,
                                           i64, f32p, vp]
    lib.nvfp4_rmsnorm_backward_workspace.restype = i64
    lib.nvfp4_rmsnorm_backward_workspace.argtypes = [i64, i64]
    lib.nvfp4_int8_quantize.restype = c_int
    lib.nvfp4_int8_quantize.argtypes = [vp, c_int, i64, i64, f32p, vp, f32p, vp]
    lib.nvfp4_int8_quantize_rowcol.restype = c_int
    lib.nvfp4_int8_quantize_rowcol.argtypes = [vp, c_int, i64, i64, f32p, f32p, vp, vp, f32p, vp]
    lib.nvfp4_int8_gemm.restype = c_int
    lib.nvfp4_int8_gemm.argtypes = [vp, c_int, f32p, vp, c_int, f32p, i64, i64, i64, vp, c_int, c_int, vp,
                                    vp, vp, c_int, f32p, vp]
    lib.nvfp4_layernorm.restype = c_int
    lib.nvfp4_layernorm.argtypes = [vp, vp, c_int, vp, vp, c_int, c_f, i64, i64, vp, vp, c_int, f32p, f32p,
                                    c_int, u8p, u8p, f32p, c_f, f32p, vp]
    lib.nvfp4_layernorm_backward.restype = c_int
    lib.nvfp4_layernorm_backward.argtypes = [vp, vp, c_int, vp, c_int, f32p, f32p, vp, i64, i64, vp, f32p,
                                             f32p, vp, i64, f32p, vp]
    lib.nvfp4_layernorm_backward_workspace.restype = i64
    lib.nvfp4_layernorm_backward_workspace.argtypes = [i64, i64]
    lib.nvfp4_cache_write.restype = c_int
    lib.nvfp4_cache_write.argtypes = [vp, i64, vp, i64, c_int, i64, i64, i64, c_int, c_f, i64, i64, vp, vp,
                                      f32p, vp, vp, f32p, vp, i64, i64, vp, vp, f32p, vp]
    lib.nvfp4_cache_read.restype = c_int
    lib.nvfp4_cache_read.argtypes = [vp, vp, f32p, vp, vp, f32p, c_int, c_f, i64, i64, vp, i64, i64, vp, vp,
                                     i64, i64, i64, vp, i64, vp, i64, c_int, f32p, vp]
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().nvfp4_status_string(int(status)).decode()


def nvfp4_status_string(status: int) -> str:
    return status_string(status)


# ----------------------------------------------------------------- marshalling
def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return NVFP4_BF16
    if t.dtype == torch.float32:
        return NVFP4_FP32
    raise TypeError(f"expected bfloat16 or float32, got {t.dtype}")


def _dev(t: Optional[torch.Tensor], name: str, dtypes, numel: Optional[int] = None,
         device: Optional[torch.device] = None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} entries, got {t.numel()}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


_SCALE_DTYPES = (torch.uint8, torch.float8_e4m3fn)
_F32 = (torch.float32,)


def _check(fn: str, status: int):
    if status != NVFP4_OK:
        raise Nvfp4Error(fn, status)


# ------------------------------------------------------------------ entry points
def nvfp4_amax_path(in_dtype: int, M: int, K: int, want_row: bool, want_col: bool,
                    flags: int = 0) -> int:
    return int(load_library().nvfp4_amax_path(in_dtype, M, K, int(want_row), int(want_col), flags))


def nvfp4_amax_rowcol(x: torch.Tensor, row_amax: Optional[torch.Tensor] = None,
                      col_amax: Optional[torch.Tensor] = None,
                      tensor_amax: Optional[torch.Tensor] = None,
                      noop: Optional[torch.Tensor] = None, flags: int = 0, stream=None) -> None:
    """row_amax [M], col_amax [K], tensor_amax [1] (float32, any subset)."""
    lib = load_library()
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    _dev(x, "x", (torch.bfloat16, torch.float32))
    M, K = x.shape
    dev = x.device
    _dev(row_amax, "row_amax", _F32, M, dev)
    _dev(col_amax, "col_amax", _F32, K, dev)
    _dev(tensor_amax, "tensor_amax", _F32, 1, dev)
    _dev(noop, "noop", _F32, 1, dev)
    st = lib.nvfp4_amax_rowcol(_ptr(x), _dtype_code(x), M, K, _ptr(row_amax), _ptr(col_amax),
                               _ptr(tensor_amax), _ptr(noop), flags, _stream(stream, dev))
    _check("nvfp4_amax_rowcol", st)


def nvfp4_check_group_end(group_end: torch.Tensor, M: int) -> int:
    """Host-side validation of group ends held in host memory (int64 CPU
    tensor); returns the C status (NVFP4_OK or NVFP4_ERR_ARG)."""
    if not isinstance(group_end, torch.Tensor) or group_end.is_cuda:
        raise ValueError("group_end must be a host (CPU) tensor")
    if group_end.dtype != torch.int64 or not group_end.is_contiguous():
        raise TypeError("group_end must be a contiguous int64 tensor")
    return int(load_library().nvfp4_check_group_end(ctypes.c_void_p(group_end.data_ptr()),
                                                    group_end.numel(), int(M)))


def nvfp4_group_amax_expand(row_amax: torch.Tensor, group_end: torch.Tensor,
                            status: Optional[torch.Tensor] = None,
                            noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """group_end: an int64 device tensor (validated on the device when a
    status [1] int32 device tensor is given), or an int64 CPU tensor, which
    is validated on the host (Nvfp4Error with NVFP4_ERR_ARG when a group
    boundary is misaligned) and then copied to the device."""
    lib = load_library()
    _dev(row_amax, "row_amax", _F32)
    dev = row_amax.device
    if isinstance(group_end, torch.Tensor) and not group_end.is_cuda:
        _check("nvfp4_check_group_end", nvfp4_check_group_end(group_end, row_amax.numel()))
        group_end = group_end.to(dev)
    _dev(group_end, "group_end", (torch.int64,), None, dev)
    _dev(status, "status", (torch.int32,), 1, dev)
    _dev(noop, "noop", _F32, 1, dev)
    st = lib.nvfp4_group_amax_expand(_ptr(row_amax), row_amax.numel(), _ptr(group_end),
                                     group_end.numel(), _ptr(status), _ptr(noop),
                                     _stream(stream, dev))
    _check("nvfp4_group_amax_expand", st)


def _amax_numel(mode: int, lines: int, length: int) -> int:
    return {NVFP4_AMAX_TENSOR: 1, NVFP4_AMAX_LINE: lines, NVFP4_AMAX_ROWGROUP: length}.get(mode, -1)


def nvfp4_quantize_transpose(x: torch.Tensor, row_mode: int, row_amax: Optional[torch.Tensor],
                             col_mode: int, col_amax: Optional[torch.Tensor], bound: float,
                             q_row: Optional[torch.Tensor], s_row: Optional[torch.Tensor],
                             q_col: Optional[torch.Tensor], s_col: Optional[torch.Tensor],
                             noop: Optional[torch.Tensor] = None, stream=None) -> None:
    _quantize("nvfp4_quantize_transpose", x, row_mode, row_amax, col_mode, col_amax, bound,
              q_row, s_row, q_col, s_col, noop, stream)


def nvfp4_quantize_rowcol(x: torch.Tensor, row_amax: torch.Tensor, col_amax: torch.Tensor,
                          bound: float, q_row: torch.Tensor, s_row: torch.Tensor,
                          q_col: torch.Tensor, s_col: torch.Tensor,
                          noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """The whole row-scaled quantize in one call: row_amax [M] and col_amax
    [K] are written, then both copies (mode LINE)."""
    lib = load_library()
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    _dev(x, "x", (torch.bfloat16, torch.float32))
    M, K = x.shape
    dev = x.device
    _dev(row_amax, "row_amax", _F32, M, dev)
    _dev(col_amax, "col_amax", _F32, K, dev)
    _dev(q_row, "q_row", (torch.uint8,), M * ((K + 1) // 2), dev)
    _dev(s_row, "s_row", _SCALE_DTYPES, M * ((K + 15) // 16), dev)
    _dev(q_col, "q_col", (torch.uint8,), K * ((M + 1) // 2), dev)
    _dev(s_col, "s_col", _SCALE_DTYPES, K * ((M + 15) // 16), dev)
    _dev(noop, "noop", _F32, 1, dev)
    st = lib.nvfp4_quantize_rowcol(_ptr(x), _dtype_code(x), M, K, ctypes.c_float(bound),
                                   _ptr(row_amax), _ptr(col_amax), _ptr(q_row), _ptr(s_row),
                                   _ptr(q_col), _ptr(s_col), _ptr(noop), _stream(stream, dev))
    _check("nvfp4_quantize_rowcol", st)


def nvfp4_quantize_4over6(x: torch.Tensor, row_mode: int, row_amax: Optional[torch.Tensor],
                          col_mode: int, col_amax: Optional[torch.Tensor], bound: float,
                          q_row: Optional[torch.Tensor], s_row: Optional[torch.Tensor],
                          q_col: Optional[torch.Tensor], s_col: Optional[torch.Tensor],
                          noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """nvfp4_quantize_transpose with four-over-six block scales."""
    _quantize("nvfp4_quantize_4over6", x, row_mode, row_amax, col_mode, col_amax, bound,
              q_row, s_row, q_col, s_col, noop, stream)


def _quantize(name, x, row_mode, row_amax, col_mode, col_amax, bound, q_row, s_row, q_col, s_col,
              noop, stream) -> None:
    lib = load_library()
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    _dev(x, "x", (torch.bfloat16, torch.float32))
    M, K = x.shape
    dev = x.device
    if q_row is not None:
        _dev(row_amax, "row_amax", _F32, _amax_numel(row_mode, M, K), dev)
        _dev(q_row, "q_row", (torch.uint8,), M * ((K + 1) // 2), dev)
        _dev(s_row, "s_row", _SCALE_DTYPES, M * ((K + 15) // 16), dev)
    if q_col is not None:
        # ROWGROUP: the transposed lines' blocks index an [M] per-row vector
        _dev(col_amax, "col_amax", _F32, _amax_numel(col_mode, K, M), dev)
        _dev(q_col, "q_col", (torch.uint8,), K * ((M + 1) // 2), dev)
        _dev(s_col, "s_col", _SCALE_DTYPES, K * ((M + 15) // 16), dev)
    _dev(noop, "noop", _F32, 1, dev)
    st = getattr(lib, name)(_ptr(x), _dtype_code(x), M, K, row_mode, _ptr(row_amax), col_mode,
                            _ptr(col_amax), ctypes.c_float(bound), _ptr(q_row), _ptr(s_row),
                            _ptr(q_col), _ptr(s_col), _ptr(noop), _stream(stream, dev))
    _check(name, st)


def nvfp4_quantize_2d(x: torch.Tensor, tensor_amax: torch.Tensor, bound: float,
                      q_row: Optional[torch.Tensor], s_row: Optional[torch.Tensor],
                      q_col: Optional[torch.Tensor], s_col: Optional[torch.Tensor],
                      noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """x [M, K] with 16 x 16 tile scales under the per-tensor amax tensor_amax [1]."""
    lib = load_library()
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    _dev(x, "x", (torch.bfloat16, torch.float32))
    M, K = x.shape
    dev = x.device
    _dev(tensor_amax, "tensor_amax", _F32, 1, dev)
    if q_row is not None:
        _dev(q_row, "q_row", (torch.uint8,), M * ((K + 1) // 2), dev)
        _dev(s_row, "s_row", _SCALE_DTYPES, M * ((K + 15) // 16), dev)
    if q_col is not None:
        _dev(q_col, "q_col", (torch.uint8,), K * ((M + 1) // 2), dev)
        _dev(s_col, "s_col", _SCALE_DTYPES, K * ((M + 15) // 16), dev)
    _dev(noop, "noop", _F32, 1, dev)
    st = lib.nvfp4_quantize_2d(_ptr(x), _dtype_code(x), M, K, _ptr(tensor_amax),
                               ctypes.c_float(bound), _ptr(q_row), _ptr(s_row), _ptr(q_col),
                               _ptr(s_col), _ptr(noop), _stream(stream, dev))
    _check("nvfp4_quantize_2d", st)


def padded_rows_max(T: int, G: int, align: int) -> int:
    """Rows the padded layout of T tokens in G groups can need at most."""
    return -(-(T + G * (align - 1)) // align) * align


def nvfp4_quantize_grouped(x: torch.Tensor, group_rows: torch.Tensor, align: int, M_out: int,
                           bound: float, row_amax: torch.Tensor,
                           q_row: Optional[torch.Tensor], s_row: Optional[torch.Tensor],
                           q_col: Optional[torch.Tensor], s_col: Optional[torch.Tensor],
                           noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """Grouped tokens x [T, K] (group sizes in the device int64 tensor
    group_rows [G]) quantized into the padded [M_out, K] layout."""
    lib = load_library()
    if x.dim() != 2:
        raise ValueError("x must be 2-D [T, K]")
    _dev(x, "x", (torch.bfloat16, torch.float32))
    T, K = x.shape
    dev = x.device
    _dev(group_rows, "group_rows", (torch.int64,), None, dev)
    _dev(row_amax, "row_amax", _F32, M_out, dev)
    if q_row is not None:
        _dev(q_row, "q_row", (torch.uint8,), M_out * ((K + 1) // 2), dev)
        _dev(s_row, "s_row", _SCALE_DTYPES, M_out * ((K + 15) // 16), dev)
    if q_col is not None:
        _dev(q_col, "q_col", (torch.uint8,), K * ((M_out + 1) // 2), dev)
        _dev(s_col, "s_col", _SCALE_DTYPES, K * ((M_out + 15) // 16), dev)
    _dev(noop, "noop", _F32, 1, dev)
    st = lib.nvfp4_quantize_grouped(_ptr(x), _dtype_code(x), T, K, _ptr(group_rows),
                                    group_rows.numel(), int(align), int(M_out),
                                    ctypes.c_float(bound), _ptr(row_amax), _ptr(q_row),
                                    _ptr(s_row), _ptr(q_col), _ptr(s_col), _ptr(noop),
                                    _stream(stream, dev))
    _check("nvfp4_quantize_grouped", st)


def nvfp4_quantize_dequantize(x: torch.Tensor, row_mode: int, row_amax: torch.Tensor,
                              bound: float, y: torch.Tensor, q_row: Optional[torch.Tensor] = None,
                              s_row: Optional[torch.Tensor] = None,
                              noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """Rowwise codes of x [M, K] (optional) and their dequantization y [M, K]
    (bfloat16 or float32) in one pass."""
    lib = load_library()
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    _dev(x, "x", (torch.bfloat16, torch.float32))
    M, K = x.shape
    dev = x.device
    _dev(row_amax, "row_amax", _F32, _amax_numel(row_mode, M, K), dev)
    _dev(y, "y", (torch.bfloat16, torch.float32), M * K, dev)
    if q_row is not None:
        _dev(q_row, "q_row", (torch.uint8,), M * ((K + 1) // 2), dev)
        _dev(s_row, "s_row", _SCALE_DTYPES, M * ((K + 15) // 16), dev)
    _dev(noop, "noop", _F32, 1, dev)
    st = lib.nvfp4_quantize_dequantize(_ptr(x), _dtype_code(x), M, K, row_mode, _ptr(row_amax),
                                       ctypes.c_float(bound), _ptr(q_row), _ptr(s_row), _ptr(y),
                                       _dtype_code(y), _ptr(noop), _stream(stream, dev))
    _check("nvfp4_quantize_dequantize", st)


def nvfp4_dequantize(q: torch.Tensor, sc: torch.Tensor, R: int, C: int, amax_mode: int,
                     amax: torch.Tensor, bound: float, y: torch.Tensor,
                     noop: Optional[torch.Tensor] = None, stream=None) -> None:
    lib = load_library()
    _dev(q, "q", (torch.uint8,), R * ((C + 1) // 2))
    dev = q.device
    _dev(sc, "sc", _SCALE_DTYPES, R * ((C + 15) // 16), dev)
    _dev(amax, "amax", _F32, _amax_numel(amax_mode, R, C), dev)
    _dev(y, "y", (torch.bfloat16, torch.float32), R * C, dev)
    _dev(noop, "noop", _F32, 1, dev)
    st = lib.nvfp4_dequantize(_ptr(q), _ptr(sc), R, C, amax_mode, _ptr(amax),
                              ctypes.c_float(bound), _ptr(y), _dtype_code(y), _ptr(noop),
                              _stream(stream, dev))
    _check("nvfp4_dequantize", st)


# ------------------------------------------ product, norm and their gradients
# These run per layer and per token, so their marshalling is lean: one pass
# over a tensor's properties, plain integers to C.
_OUT_CODES = {torch.bfloat16: NVFP4_BF16, torch.float32: NVFP4_FP32}
_U8 = (torch.uint8,)


def _arg(t, name: str, dtypes, numel: int, dev) -> Optional[int]:
    """The device address of an optional tensor argument, checked."""
    if t is None:
        return None
    try:
        if (t.dtype in dtypes and t.numel() == numel and t.get_device() == dev.index
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, name, dtypes, numel, dev)
    return t.data_ptr()


def _first(t, name: str, dtypes) -> torch.device:
    """The device of the argument that decides it for the others."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    return t.device


def _raw_stream(stream, dev) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev.index)
    return stream.cuda_stream


def _workspace(ws: Optional[torch.Tensor], need: int, dev, stream):
    """(tensor, address, bytes) of the workspace: the caller's (any dtype), or
    one from torch's allocator. That one comes from the pool of the stream the
    call runs on: what used the block before, and what takes it after, is in
    that stream's order. (A block of the current stream's pool could still be
    in use by work queued there.)"""
    if need <= 0:
        return None, None, 0
    if ws is None:
        if stream is None:
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            with torch.cuda.stream(stream):
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
    if not ws.is_cuda or ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    size = ws.numel() * ws.element_size()
    if size < need:
        raise ValueError(f"workspace must have {need} bytes, got {size}")
    return ws, ws.data_ptr(), size


def nvfp4_gemm(a: torch.Tensor, a_scale: Optional[torch.Tensor], a_mode: int, a_amax: torch.Tensor,
               a_bound: float, b: torch.Tensor, b_scale: torch.Tensor, b_mode: int,
               b_amax: torch.Tensor, b_bound: float, M: int, N: int, K: int, y: torch.Tensor,
               bias: Optional[torch.Tensor] = None, act: int = NVFP4_ACT_NONE,
               residual: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
               noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """y [M, N] = act(A B^T + bias) + residual of packed operands.

    a: uint8 codes [M, ceil(K/2)] with a_scale [M, ceil(K/16)] (NVFP4), or
    float8_e4m3fn [M, K] with a_scale None (8-bit lines). b: the N lines (2 N
    for NVFP4_ACT_SWIGLU: gate lines, then up lines), NVFP4. y, z and residual
    share y's dtype (bfloat16 or float32); bias is bfloat16 or float32."""
    lib = _lib or load_library()
    dev = _first(a, "a", (torch.uint8, torch.float8_e4m3fn))
    fmt = NVFP4_FMT_NVFP4 if a.dtype == torch.uint8 else NVFP4_FMT_E4M3
    if fmt == NVFP4_FMT_NVFP4 and a_scale is None:
        raise ValueError("a_scale is required for NVFP4 lines")
    if fmt == NVFP4_FMT_E4M3 and a_scale is not None:
        raise ValueError("a_scale must be None for E4M3 lines")
    out = _OUT_CODES.get(getattr(y, "dtype", None))
    if out is None:
        raise TypeError("y must be a bfloat16 or float32 tensor")
    NB = 2 * N if act == NVFP4_ACT_SWIGLU else N
    kq, ks = (K + 1) // 2, (K + 15) // 16
    same = (y.dtype,)
    st = lib.nvfp4_gemm(
        fmt, _arg(a, "a", (a.dtype,), M * (kq if fmt == NVFP4_FMT_NVFP4 else K), dev),
        _arg(a_scale, "a_scale", _SCALE_DTYPES, M * ks, dev), a_mode,
        _arg(a_amax, "a_amax", _F32, M if a_mode == NVFP4_AMAX_LINE else 1, dev), a_bound,
        _arg(b, "b", _U8, NB * kq, dev), _arg(b_scale, "b_scale", _SCALE_DTYPES, NB * ks, dev), b_mode,
        _arg(b_amax, "b_amax", _F32, NB if b_mode == NVFP4_AMAX_LINE else 1, dev), b_bound,
        M, N, K, _arg(bias, "bias", _OUT_CODES, NB, dev),
        0 if bias is None else _OUT_CODES[bias.dtype], act,
        _arg(residual, "residual", same, M * N, dev), _arg(z, "z", same, M * NB, dev),
        _arg(y, "y", same, M * N, dev), out, _arg(noop, "noop", _F32, 1, dev),
        _raw_stream(stream, dev))
    if st:
        raise Nvfp4Error("nvfp4_gemm", st)


def nvfp4_act_backward_workspace(M: int, N: int, act: int) -> int:
    """Workspace bytes of nvfp4_act_backward with dbias."""
    return load_library().nvfp4_act_backward_workspace(M, N, act)


def nvfp4_act_backward(dy: torch.Tensor, z: torch.Tensor, act: int, dz: torch.Tensor,
                       dbias: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """dz = dy * act'(z) of dy [M, N], and dbias (float32) = its sum over rows.
    z and dz have dy's shape ([M, 2 N] for NVFP4_ACT_SWIGLU) and dtype."""
    lib = _lib or load_library()
    dev = _first(dy, "dy", _OUT_CODES)
    if dy.dim() != 2:
        raise ValueError("dy must be 2-D [M, N]")
    M, N = dy.shape
    NB = 2 * N if act == NVFP4_ACT_SWIGLU else N
    same = (dy.dtype,)
    need = lib.nvfp4_act_backward_workspace(M, N, act) if dbias is not None else 0
    ws, wp, wb = _workspace(workspace, need, dev, stream)
    st = lib.nvfp4_act_backward(
        _arg(dy, "dy", same, M * N, dev), _arg(z, "z", same, M * NB, dev), _OUT_CODES[dy.dtype], M, N,
        act, _arg(dz, "dz", same, M * NB, dev), _arg(dbias, "dbias", _F32, NB, dev), wp, wb,
        _arg(noop, "noop", _F32, 1, dev), _raw_stream(stream, dev))
    if st:
        raise Nvfp4Error("nvfp4_act_backward", st)


def nvfp4_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float,
                  residual: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                  y: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                  q: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
                  row_amax: Optional[torch.Tensor] = None, bound: float = 448.0,
                  noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """h = x + residual, y = h / rms(h) * weight of x [M, K], with y's row
    amax and codes: q float8_e4m3fn [M, K] (8-bit lines), or uint8
    [M, ceil(K/2)] with s [M, ceil(K/16)] (NVFP4). Outputs not given are not
    written; rstd is what nvfp4_rmsnorm_backward takes."""
    lib = _lib or load_library()
    dev = _first(x, "x", _OUT_CODES)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = x.shape
    same = (x.dtype,)
    fmt, qn = NVFP4_FMT_NONE, 0
    if q is not None:
        if q.dtype == torch.float8_e4m3fn:
            fmt, qn = NVFP4_FMT_E4M3, M * K
        else:
            fmt, qn = NVFP4_FMT_NVFP4, M * ((K + 1) // 2)
    st = lib.nvfp4_rmsnorm(
        _arg(x, "x", same, M * K, dev), _arg(residual, "residual", same, M * K, dev),
        _OUT_CODES[x.dtype], _arg(weight, "weight", _OUT_CODES, K, dev),
        _OUT_CODES.get(getattr(weight, "dtype", None), -1), eps, M, K, _arg(h, "h", same, M * K, dev),
        _arg(y, "y", _OUT_CODES, M * K, dev), 0 if y is None else _OUT_CODES[y.dtype],
        _arg(rstd, "rstd", _F32, M, dev), fmt,
        _arg(q, "q", (torch.float8_e4m3fn, torch.uint8), qn, dev),
        _arg(s, "s", _SCALE_DTYPES, M * ((K + 15) // 16), dev),
        _arg(row_amax, "row_amax", _F32, M, dev), bound, _arg(noop, "noop", _F32, 1, dev),
        _raw_stream(stream, dev))
    if st:
        raise Nvfp4Error("nvfp4_rmsnorm", st)


def nvfp4_rmsnorm_backward_workspace(M: int, K: int) -> int:
    """Workspace bytes of nvfp4_rmsnorm_backward with dweight."""
    return load_library().nvfp4_rmsnorm_backward_workspace(M, K)


def nvfp4_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                           rstd: torch.Tensor, dx: torch.Tensor,
                           dweight: Optional[torch.Tensor] = None,
                           dres: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None,
                           noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """dx [M, K] and dweight [K] (float32) of nvfp4_rmsnorm from dy [M, K], the
    saved h and rstd; dres, the gradient that reaches h by other ways, is added
    to dx."""
    lib = _lib or load_library()
    dev = _first(dy, "dy", _OUT_CODES)
    if dy.dim() != 2:
        raise ValueError("dy must be 2-D [M, K]")
    M, K = dy.shape
    same = (dy.dtype,)
    need = lib.nvfp4_rmsnorm_backward_workspace(M, K) if dweight is not None else 0
    ws, wp, wb = _workspace(workspace, need, dev, stream)
    st = lib.nvfp4_rmsnorm_backward(
        _arg(dy, "dy", same, M * K, dev), _arg(h, "h", same, M * K, dev), _OUT_CODES[dy.dtype],
        _arg(weight, "weight", _OUT_CODES, K, dev), _OUT_CODES.get(getattr(weight, "dtype", None), -1),
        _arg(rstd, "rstd", _F32, M, dev), _arg(dres, "dres", same, M * K, dev), M, K,
        _arg(dx, "dx", same, M * K, dev), _arg(dweight, "dweight", _F32, K, dev), wp, wb,
        _arg(noop, "noop", _F32, 1, dev), _raw_stream(stream, dev))
    if st:
        raise Nvfp4Error("nvfp4_rmsnorm_backward", st)


# -------------------------------- 8-bit integers, layer norm, quantized cache
# A decode step's kernels run for a few us: _calls.so checks the tensors and calls
# the library. Where it finds something amiss it returns None, and the checks
# here, which are the same, say what.
_short = None


def _load_short():
    global _short
    load_library()
    if not os.path.exists(calls_path()):
        raise ImportError(f"{calls_path()} is missing: build it with __graft_entry__.build()")
    _short = importlib.import_module("._calls", __name__)
    return _short


_I8 = (torch.int8,)
_I32 = (torch.int32,)


def nvfp4_int8_quantize(x: torch.Tensor, row_amax: torch.Tensor, q: torch.Tensor,
                        noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """Rows of x [M, K] as 8-bit integers: row_amax [M] float32 and q [M, K] int8,
    both written; value = q * row_amax / 127."""
    st = (_short or _load_short()).int8_quantize(x, row_amax, q, noop, stream)
    if st is None:
        lib = load_library()
        dev = _first(x, "x", _OUT_CODES)
        if x.dim() != 2:
            raise ValueError("x must be 2-D [M, K]")
        M, K = x.shape
        with torch.cuda.device(dev):
            st = lib.nvfp4_int8_quantize(_arg(x, "x", (x.dtype,), M * K, dev), _OUT_CODES[x.dtype], M, K,
                                         _arg(row_amax, "row_amax", _F32, M, dev), _arg(q, "q", _I8, M * K, dev),
                                         _arg(noop, "noop", _F32, 1, dev), _raw_stream(stream, dev))
    if st:
        raise Nvfp4Error("nvfp4_int8_quantize", st)


def nvfp4_int8_quantize_rowcol(x: torch.Tensor, row_amax: torch.Tensor, col_amax: torch.Tensor,
                               q_row: torch.Tensor, q_col: torch.Tensor,
                               noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """Both copies of x [M, K] as 8-bit integers: row_amax [M] and q_row [M, K],
    col_amax [K] and q_col [K, M] (the transpose), all written."""
    st = (_short or _load_short()).int8_quantize_rowcol(x, row_amax, col_amax, q_row, q_col, noop, stream)
    if st is None:
        lib = load_library()
        dev = _first(x, "x", _OUT_CODES)
        if x.dim() != 2:
            raise ValueError("x must be 2-D [M, K]")
        M, K = x.shape
        with torch.cuda.device(dev):
            st = lib.nvfp4_int8_quantize_rowcol(
                _arg(x, "x", (x.dtype,), M * K, dev), _OUT_CODES[x.dtype], M, K,
                _arg(row_amax, "row_amax", _F32, M, dev), _arg(col_amax, "col_amax", _F32, K, dev),
                _arg(q_row, "q_row", _I8, M * K, dev), _arg(q_col, "q_col", _I8, M * K, dev),
                _arg(noop, "noop", _F32, 1, dev), _raw_stream(stream, dev))
    if st:
        raise Nvfp4Error("nvfp4_int8_quantize_rowcol", st)


def nvfp4_int8_gemm(a: torch.Tensor, a_mode: int, a_amax: torch.Tensor, b: torch.Tensor, b_mode: int,
                    b_amax: torch.Tensor, M: int, N: int, K: int, y: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, act: int = NVFP4_ACT_NONE,
                    residual: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                    noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """y [M, N] = act(A B^T + bias) + residual of 8-bit integer lines a [M, K] and
    b [N, K] (2 N lines for NVFP4_ACT_SWIGLU: gate lines, then up lines), each
    line with its amax (or one for all, NVFP4_AMAX_TENSOR). z, y, residual and
    bias as in nvfp4_gemm."""
    st = (_short or _load_short()).int8_gemm(a, a_mode, a_amax, b, b_mode, b_amax, M, N, K, y, bias, act,
                                             residual, z, noop, stream)
    if st is None:
        lib = load_library()
        dev = _first(a, "a", _I8)
        out = _OUT_CODES.get(getattr(y, "dtype", None))
        if out is None:
            raise TypeError("y must be a bfloat16 or float32 tensor")
        NB = 2 * N if act == NVFP4_ACT_SWIGLU else N
        same = (y.dtype,)
        with torch.cuda.device(dev):
            st = lib.nvfp4_int8_gemm(
                _arg(a, "a", _I8, M * K, dev), a_mode,
                _arg(a_amax, "a_amax", _F32, M if a_mode == NVFP4_AMAX_LINE else 1, dev),
                _arg(b, "b", _I8, NB * K, dev), b_mode,
                _arg(b_amax, "b_amax", _F32, NB if b_mode == NVFP4_AMAX_LINE else 1, dev),
                M, N, K, _arg(bias, "bias", _OUT_CODES, NB, dev),
                0 if bias is None else _OUT_CODES[bias.dtype], act,
                _arg(residual, "residual", same, M * N, dev), _arg(z, "z", same, M * NB, dev),
                _arg(y, "y", same, M * N, dev), out, _arg(noop, "noop", _F32, 1, dev),
                _raw_stream(stream, dev))
    if st:
        raise Nvfp4Error("nvfp4_int8_gemm", st)


_NORM_FORMATS = {torch.float8_e4m3fn: NVFP4_FMT_E4M3, torch.int8: NVFP4_FMT_INT8, torch.uint8: NVFP4_FMT_NVFP4}


def nvfp4_layernorm(x: torch.Tensor, weight: torch.Tensor, eps: float, bias: Optional[torch.Tensor] = None,
                    residual: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                    y: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                    rstd: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                    s: Optional[torch.Tensor] = None, row_amax: Optional[torch.Tensor] = None,
                    bound: float = 448.0, noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """h = x + residual, y = (h - mean) / deviation * weight + bias of x [M, K],
    with y's row amax and codes: q float8_e4m3fn or int8 [M, K] (8-bit lines), or
    uint8 [M, ceil(K/2)] with s [M, ceil(K/16)] (NVFP4). bias has weight's dtype.
    Outputs not given are not written; mean and rstd are what
    nvfp4_layernorm_backward takes."""
    st = (_short or _load_short()).layernorm(x, weight, eps, bias, residual, h, y, mean, rstd, q, s, row_amax,
                                             bound, noop, stream)
    if st is None:
        lib = load_library()
        dev = _first(x, "x", _OUT_CODES)
        if x.dim() != 2:
            raise ValueError("x must be 2-D [M, K]")
        M, K = x.shape
        same, wtype = (x.dtype,), getattr(weight, "dtype", None)
        fmt, qn = NVFP4_FMT_NONE, 0
        if q is not None:
            fmt = _NORM_FORMATS.get(q.dtype, NVFP4_FMT_NVFP4)
            qn = M * ((K + 1) // 2) if fmt == NVFP4_FMT_NVFP4 else M * K
        with torch.cuda.device(dev):
            st = lib.nvfp4_layernorm(
                _arg(x, "x", same, M * K, dev), _arg(residual, "residual", same, M * K, dev),
                _OUT_CODES[x.dtype], _arg(weight, "weight", _OUT_CODES, K, dev), _arg(bias, "bias", (wtype,), K, dev),
                _OUT_CODES.get(wtype, -1), eps, M, K, _arg(h, "h", same, M * K, dev),
                _arg(y, "y", _OUT_CODES, M * K, dev), 0 if y is None else _OUT_CODES[y.dtype],
                _arg(mean, "mean", _F32, M, dev), _arg(rstd, "rstd", _F32, M, dev), fmt,
                _arg(q, "q", tuple(_NORM_FORMATS), qn, dev),
                _arg(s, "s", _SCALE_DTYPES, M * ((K + 15) // 16), dev),
                _arg(row_amax, "row_amax", _F32, M, dev), bound, _arg(noop, "noop", _F32, 1, dev),
                _raw_stream(stream, dev))
    if st:
        raise Nvfp4Error("nvfp4_layernorm", st)


def nvfp4_layernorm_backward_workspace(M: int, K: int) -> int:
    """Workspace bytes of nvfp4_layernorm_backward with dweight or dbias."""
    return load_library().nvfp4_layernorm_backward_workspace(M, K)


def nvfp4_layernorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                             mean: torch.Tensor, rstd: torch.Tensor, dx: torch.Tensor,
                             dweight: Optional[torch.Tensor] = None,
                             dbias: Optional[torch.Tensor] = None,
                             dres: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None,
                             noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """dx [M, K], dweight [K] and dbias [K] (float32) of nvfp4_layernorm from
    dy [M, K] and the saved h, mean and rstd; dres, the gradient that reaches h by
    other ways, is added to dx."""
    st = (_short or _load_short()).layernorm_backward(dy, h, weight, mean, rstd, dx, dweight, dbias, dres,
                                                      workspace, noop, stream)
    if st is None:
        lib = load_library()
        dev = _first(dy, "dy", _OUT_CODES)
        if dy.dim() != 2:
            raise ValueError("dy must be 2-D [M, K]")
        M, K = dy.shape
        same = (dy.dtype,)
        sums = dweight is not None or dbias is not None
        need = lib.nvfp4_layernorm_backward_workspace(M, K) if sums else 0
        ws, wp, wb = _workspace(workspace, need, dev, stream)
        with torch.cuda.device(dev):
            st = lib.nvfp4_layernorm_backward(
                _arg(dy, "dy", same, M * K, dev), _arg(h, "h", same, M * K, dev), _OUT_CODES[dy.dtype],
                _arg(weight, "weight", _OUT_CODES, K, dev), _OUT_CODES.get(getattr(weight, "dtype", None), -1),
                _arg(mean, "mean", _F32, M, dev), _arg(rstd, "rstd", _F32, M, dev),
                _arg(dres, "dres", same, M * K, dev), M, K, _arg(dx, "dx", same, M * K, dev),
                _arg(dweight, "dweight", _F32, K, dev), _arg(dbias, "dbias", _F32, K, dev), wp, wb,
                _arg(noop, "noop", _F32, 1, dev), _raw_stream(stream, dev))
    if st:
        raise Nvfp4Error("nvfp4_layernorm_backward", st)


_CACHE_FORMATS = {torch.float8_e4m3fn: NVFP4_FMT_E4M3, torch.int8: NVFP4_FMT_INT8, torch.uint8: NVFP4_FMT_NVFP4}


def _rows(t, name: str, dtypes, shape, dev):
    """(address, elements from row to row) of [T, H, D] rows that may lie apart."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    T, H, D = t.shape
    st, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"each row of {name} must be contiguous")
    return t.data_ptr(), st if T > 1 else H * D


def _cache(k_q, k_s, k_amax, v_q, v_s, v_amax, D, dev):
    """Checked cache buffers: (format, pages, page_size, H, the six addresses)."""
    fmt = _CACHE_FORMATS.get(getattr(k_q, "dtype", None))
    if fmt is None:
        raise TypeError("k_q must be a uint8 (NVFP4), float8_e4m3fn or int8 tensor")
    if not isinstance(k_amax, torch.Tensor) or k_amax.dim() != 3:
        raise ValueError("k_amax must be 3-D [pages, page_size, H]")
    pages, size, H = k_amax.shape
    lines = pages * size * H
    width, blocks = ((D + 1) // 2, (D + 15) // 16) if fmt == NVFP4_FMT_NVFP4 else (D, 0)
    addr = []
    for n, q, s, a in (("k", k_q, k_s, k_amax), ("v", v_q, v_s, v_amax)):
        if q is None and (s is not None or a is not None or n == "k"):
            raise ValueError(f"{n}_q is required")
        if q is not None and a is None:
            raise ValueError(f"{n}_amax is required")
        if q is not None and (s is not None) != (fmt == NVFP4_FMT_NVFP4):
            raise ValueError(f"{n}_s is for NVFP4 lines, and they need it")
        addr += [_arg(q, n + "_q", (k_q.dtype,), lines * width, dev),
                 _arg(s, n + "_s", _SCALE_DTYPES, lines * blocks, dev), _arg(a, n + "_amax", _F32, lines, dev)]
    return fmt, pages, size, H, addr


def _sequences(table, starts, first, dev):
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be 2-D [B, columns]")
    B, cols = table.shape
    return (_arg(table, "table", _I32, B * cols, dev), B, cols, _arg(starts, "starts", _I32, B + 1, dev),
            _arg(first, "first", _I32, B, dev))


def nvfp4_cache_write(k: torch.Tensor, v: Optional[torch.Tensor], k_q: torch.Tensor,
                      k_s: Optional[torch.Tensor], k_amax: torch.Tensor, v_q: Optional[torch.Tensor],
                      v_s: Optional[torch.Tensor], v_amax: Optional[torch.Tensor], table: torch.Tensor,
                      starts: torch.Tensor, first: Optional[torch.Tensor] = None, bound: float = 448.0,
                      noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """Keys and values of new tokens, k and v [T, H, D] (rows may lie apart, as
    slices of a fused projection do; v None: keys alone), quantized into pages:
    amax [pages, page_size, H] float32; q [pages, page_size, H, D] float8_e4m3fn
    or int8, or uint8 [.., ceil(D/2)] with s [.., ceil(D/16)] (NVFP4).

    Sequence b has the rows starts[b] .. starts[b + 1] - 1 and they take its
    positions from first[b] (0 without first) on; position n lies at place
    n % page_size of page table[b, n // page_size]. table [B, columns], starts
    [B + 1] and first [B] are int32 device tensors. Tokens without a page are
    skipped."""
    st = (_short or _load_short()).cache_write(k, v, k_q, k_s, k_amax, v_q, v_s, v_amax, table, starts, first,
                                               bound, noop, stream)
    if st is None:
        lib = load_library()
        dev = _first(k, "k", _OUT_CODES)
        if k.dim() != 3:
            raise ValueError("k must be 3-D [T, H, D]")
        T, H, D = k.shape
        fmt, pages, size, heads, buf = _cache(k_q, k_s, k_amax, v_q, v_s, v_amax, D, dev)
        if heads != H or (v is None) != (v_q is None):
            raise ValueError("k and v must match the cache's heads and buffers")
        kp, ks = _rows(k, "k", (k.dtype,), k.shape, dev)
        vp, vs = _rows(v, "v", (k.dtype,), k.shape, dev)
        tp, B, cols, sp, fp = _sequences(table, starts, first, dev)
        with torch.cuda.device(dev):
            st = lib.nvfp4_cache_write(kp, ks, vp, vs, _OUT_CODES[k.dtype], T, H, D, fmt, bound, pages, size, *buf,
                                       tp, B, cols, sp, fp, _arg(noop, "noop", _F32, 1, dev), _raw_stream(stream, dev))
    if st:
        raise Nvfp4Error("nvfp4_cache_write", st)


def nvfp4_cache_read(k: torch.Tensor, v: Optional[torch.Tensor], k_q: torch.Tensor,
                     k_s: Optional[torch.Tensor], k_amax: torch.Tensor, v_q: Optional[torch.Tensor],
                     v_s: Optional[torch.Tensor], v_amax: Optional[torch.Tensor], table: torch.Tensor,
                     starts: torch.Tensor, first: Optional[torch.Tensor] = None, bound: float = 448.0,
                     noop: Optional[torch.Tensor] = None, stream=None) -> None:
    """The cached tokens of each sequence as values, into rows starts[b] ..
    starts[b + 1] - 1 of k and v [T, H, D] (bfloat16 or float32): its positions
    from first[b] on. Arguments as nvfp4_cache_write; rows of no sequence stay as
    they are, tokens without a page read as zeros."""
    st = (_short or _load_short()).cache_read(k, v, k_q, k_s, k_amax, v_q, v_s, v_amax, table, starts, first,
                                              bound, noop, stream)
    if st is None:
        lib = load_library()
        dev = _first(k, "k", _OUT_CODES)
        if k.dim() != 3:
            raise ValueError("k must be 3-D [T, H, D]")
        T, H, D = k.shape
        fmt, pages, size, heads, buf = _cache(k_q, k_s, k_amax, v_q, v_s, v_amax, D, dev)
        if heads != H or (v is None) != (v_q is None):
            raise ValueError("k and v must match the cache's heads and buffers")
        kp, ks = _rows(k, "k", (k.dtype,), k.shape, dev)
        vp, vs = _rows(v, "v", (k.dtype,), k.shape, dev)
        tp, B, cols, sp, fp = _sequences(table, starts, first, dev)
        with torch.cuda.device(dev):
            st = lib.nvfp4_cache_read(*buf, fmt, bound, pages, size, tp, B, cols, sp, fp, T, H, D, kp, ks, vp, vs,
                                      _OUT_CODES[k.dtype], _arg(noop, "noop", _F32, 1, dev), _raw_stream(stream, dev))
    if st:
        raise Nvfp4Error("nvfp4_cache_read", st)


# --------------------------------------------------------------- conveniences
def empty_outputs(M: int, K: int, device, rowwise: bool = True, colwise: bool = True) -> dict:
    """Allocate the packed output buffers for an M x K input."""
    out = {}
    if rowwise:
        out["q_row"] = torch.empty(M, (K + 1) // 2, dtype=torch.uint8, device=device)
        out["s_row"] = torch.empty(M, (K + 15) // 16, dtype=torch.uint8, device=device)
    if colwise:
        out["q_col"] = torch.empty(K, (M + 1) // 2, dtype=torch.uint8, device=device)
        out["s_col"] = torch.empty(K, (M + 15) // 16, dtype=torch.uint8, device=device)
    return out
