"""NVFP4 quantize / dequantize on GB300 (sm_103a) -- Python binding of libnvfp4.

Thin ctypes layer over the C ABI declared in ``include/nvfp4.h``: the functions
keep the C names and only marshal arguments (torch tensors -> device pointers,
the current torch stream -> cudaStream_t).  Every step of the computation runs
in the library's CUDA kernels; there is no CPU or PyTorch fallback, and
importing a function without the compiled library raises.

PyTorch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes as C
import os
import platform
from array import array
from contextlib import nullcontext
from dataclasses import dataclass
from typing import Optional

import torch

__all__ = [
    "NVFP4_OK", "NVFP4_IN_BF16", "NVFP4_IN_FP32", "NVFP4_OUT_BF16", "NVFP4_OUT_FP32",
    "NVFP4_PER_TENSOR", "NVFP4_ROW_SCALED", "NVFP4_DEVICE_TIMEOUT", "NVFP4_DEVICE_BAD_GROUPS",
    "Config", "Out", "NVFP4Error", "load_library", "library_path",
    "nvfp4_amax", "nvfp4_quantize_rowwise", "nvfp4_quantize_columnwise", "nvfp4_quantize_both",
    "nvfp4_dequantize", "nvfp4_grouped_amax", "nvfp4_grouped_quantize_rowwise",
    "nvfp4_grouped_quantize_rowwise_padded", "nvfp4_grouped_quantize_columnwise",
    "nvfp4_last_error", "nvfp4_device_status", "nvfp4_selftest_convert",
    "nvfp4_selftest_wait_timeout", "nvfp4_selftest_scale_division",
    "nvfp4_gemm_workspace_size", "nvfp4_gemm", "nvfp4_gemm_static_ws", "Operand",
    "nvfp4_grouped_gemm_workspace_size", "nvfp4_grouped_gemm", "nvfp4_grouped_gemm_wgrad",
    "NVFP4_GEMM_STATIC_WS_BYTES", "alloc_out", "EXPORTED_SYMBOLS", "nvfp4_rht16",
    "nvfp4_quantize_columnwise_rht", "nvfp4_quantize_both_rht",
    "nvfp4_grouped_quantize_columnwise_rht",
    "NVFP4_ACT_NONE", "NVFP4_ACT_RELU", "NVFP4_ACT_GELU", "NVFP4_ACT_SILU", "Fp8Out",
    "NVFP4_RMSNORM_MAX_COLS", "nvfp4_add_rmsnorm", "nvfp4_add_rmsnorm_backward",
    "nvfp4_add_rmsnorm_backward_workspace_size", "nvfp4_gemm_bias_act",
    "nvfp4_gemm_bias_act_workspace_size", "nvfp4_bias_act_backward",
    "nvfp4_bias_act_backward_workspace_size", "nvfp4_grad_norm", "nvfp4_clip_grad_norm",
    "nvfp4_clip_grad_norm_workspace_size",
]

NVFP4_OK = 0
NVFP4_ERR_INVALID = 1
NVFP4_ERR_UNSUPPORTED = 2
NVFP4_ERR_CUDA = 3
NVFP4_ERR_TIMEOUT = 4
NVFP4_IN_BF16 = 0
NVFP4_IN_FP32 = 1
NVFP4_OUT_BF16 = 0
NVFP4_OUT_FP32 = 1
NVFP4_PER_TENSOR = 0
NVFP4_ROW_SCALED = 1
NVFP4_DEVICE_TIMEOUT = 1
NVFP4_DEVICE_BAD_GROUPS = 2
NVFP4_GEMM_STATIC_WS_BYTES = 64 << 20
NVFP4_ACT_NONE = 0
NVFP4_ACT_RELU = 1
NVFP4_ACT_GELU = 2
NVFP4_ACT_SILU = 3
NVFP4_RMSNORM_MAX_COLS = 32768

EXPORTED_SYMBOLS = (
    "nvfp4_amax", "nvfp4_quantize_rowwise", "nvfp4_quantize_columnwise", "nvfp4_quantize_both",
    "nvfp4_dequantize", "nvfp4_grouped_amax", "nvfp4_grouped_quantize_rowwise",
    "nvfp4_grouped_quantize_rowwise_padded", "nvfp4_grouped_quantize_columnwise",
    "nvfp4_last_error", "nvfp4_device_status", "nvfp4_selftest_convert",
    "nvfp4_selftest_wait_timeout", "nvfp4_selftest_scale_division",
    "nvfp4_gemm_workspace_size", "nvfp4_gemm", "nvfp4_gemm_static_ws",
    "nvfp4_grouped_gemm_workspace_size", "nvfp4_grouped_gemm", "nvfp4_grouped_gemm_wgrad",
    "nvfp4_rht16", "nvfp4_quantize_columnwise_rht", "nvfp4_quantize_both_rht",
    "nvfp4_grouped_quantize_columnwise_rht",
    "nvfp4_add_rmsnorm", "nvfp4_add_rmsnorm_backward",
    "nvfp4_add_rmsnorm_backward_workspace_size", "nvfp4_gemm_bias_act",
    "nvfp4_gemm_bias_act_workspace_size", "nvfp4_bias_act_backward",
    "nvfp4_bias_act_backward_workspace_size", "nvfp4_grad_norm", "nvfp4_clip_grad_norm",
    "nvfp4_clip_grad_norm_workspace_size",
)

_HERE = os.path.dirname(os.path.abspath(__file__))


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"nvfp4 status {status}: {message}")
        self.status = status


class Config(C.Structure):
    """nvfp4_config: mode (PER_TENSOR / ROW_SCALED), bound (448 or 256),
    four_over_six (0/1), block_2d (0: 1x16, 1: 16x16)."""
    _fields_ = [("mode", C.c_int32), ("bound", C.c_float), ("four_over_six", C.c_int32),
                ("block_2d", C.c_int32)]


class _COut(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("amax", C.c_void_p),
                ("amax_in", C.c_void_p)]


@dataclass
class Out:
    """One output direction: codes [lines][ceil(n/2)] uint8, scales
    [lines][ceil(n/16)] uint8, amax [lines] or [1] float32, optional amax_in."""
    codes: torch.Tensor
    scales: torch.Tensor
    amax: torch.Tensor
    amax_in: Optional[torch.Tensor] = None

    def _c(self) -> _COut:
        return _COut(_ptr(self.codes), _ptr(self.scales), _ptr(self.amax), _ptr(self.amax_in))

    def as_operand(self, mode: int, bound: float) -> "Operand":
        return Operand(self.codes, self.scales, self.amax, mode, bound)


def library_path() -> str:
    return os.path.join(_HERE, f"libnvfp4_{platform.machine()}.so")


_lib = None


def load_library():
    """Load libnvfp4 (raises if it has not been built: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libnvfp4 is not built ({path} missing); run "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = C.CDLL(path)
    vp, i32, i64, f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_float
    sig = {
        "nvfp4_amax": [vp, i32, i64, i64, vp, vp, vp, vp, vp],
        "nvfp4_quantize_rowwise": [vp, i32, i64, i64, vp, vp, vp, vp],
        "nvfp4_quantize_columnwise": [vp, i32, i64, i64, vp, vp, vp, vp],
        "nvfp4_quantize_both": [vp, i32, i64, i64, vp, vp, vp, vp, vp],
        "nvfp4_dequantize": [vp, vp, vp, i32, i64, i64, f32, vp, i32, vp],
        "nvfp4_grouped_amax": [vp, i32, i64, i64, vp, i32, vp, vp, vp, vp],
        "nvfp4_grouped_quantize_rowwise": [vp, i32, i64, i64, vp, i32, vp, vp, vp, vp, vp],
        "nvfp4_grouped_quantize_rowwise_padded": [vp, i32, i64, i64, vp, vp, i32, i64, vp, vp,
                                                  vp, vp, vp],
        "nvfp4_grouped_quantize_columnwise": [vp, i32, i64, i64, vp, i32, vp, vp, vp, vp],
        "nvfp4_device_status": [C.POINTER(C.c_int32), i32],
        "nvfp4_selftest_convert": [vp, i64, vp, vp, vp],
        "nvfp4_selftest_wait_timeout": [i64, vp, vp],
        "nvfp4_selftest_scale_division": [vp, i64, vp, vp],
        "nvfp4_gemm_workspace_size": [i64, i64, i64, C.POINTER(C.c_uint64)],
        "nvfp4_gemm": [vp, vp, i64, i64, i64, vp, i32, vp, C.c_uint64, vp],
        "nvfp4_gemm_static_ws": [vp, vp, i64, i64, i64, vp, i32, vp],
        "nvfp4_grouped_gemm_workspace_size": [i64, i64, i64, i32, C.POINTER(C.c_uint64)],
        "nvfp4_grouped_gemm": [vp, vp, vp, i32, i64, i64, i64, vp, i32, vp, C.c_uint64, vp],
        "nvfp4_grouped_gemm_wgrad": [vp, vp, vp, i32, i64, i64, i64, vp, i32, vp, C.c_uint64,
                                     vp],
        "nvfp4_rht16": [vp, i32, i64, i64, C.c_uint32, vp, vp],
        "nvfp4_quantize_columnwise_rht": [vp, i32, i64, i64, C.c_uint32, vp, vp, vp, C.c_uint64,
                                          vp, vp],
        "nvfp4_quantize_both_rht": [vp, i32, i64, i64, C.c_uint32, vp, vp, vp, vp, vp],
        "nvfp4_grouped_quantize_columnwise_rht": [vp, i32, i64, i64, vp, i32, C.c_uint32, vp, vp,
                                                  vp, vp],
        "nvfp4_add_rmsnorm": [vp, vp, i32, vp, i32, i64, i64, f32, vp, vp, vp, vp, vp, vp, vp],
        "nvfp4_add_rmsnorm_backward_workspace_size": [i64, i64, C.POINTER(C.c_uint64)],
        "nvfp4_add_rmsnorm_backward": [vp, vp, vp, i32, vp, i32, vp, i64, i64, vp, vp, vp,
                                       C.c_uint64, vp],
        "nvfp4_gemm_bias_act_workspace_size": [i64, i64, i64, C.POINTER(C.c_uint64)],
        "nvfp4_gemm_bias_act": [vp, vp, i64, i64, i64, vp, vp, i32, vp, C.c_uint64, vp],
        "nvfp4_bias_act_backward_workspace_size": [i64, i64, C.POINTER(C.c_uint64)],
        "nvfp4_bias_act_backward": [vp, vp, i32, i32, i64, i64, vp, vp, vp, vp, vp, C.c_uint64,
                                    vp],
        "nvfp4_clip_grad_norm_workspace_size": [C.POINTER(C.c_uint64)],
        "nvfp4_grad_norm": [vp, i32, vp, vp, C.c_uint64, vp],
        "nvfp4_clip_grad_norm": [vp, i32, f32, vp, vp, C.c_uint64, vp],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = C.c_int
    L.nvfp4_last_error.argtypes = []
    L.nvfp4_last_error.restype = C.c_char_p
    _lib = L
    return L


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _current_raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# The handle alone where this torch has a call for it (a Stream object costs as much as the
# launch of a small kernel); it is not part of torch's interface, so a torch without it is served
# by the one above.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_raw_stream)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _workspace(workspace: Optional[torch.Tensor], need: int, device, stream):
    """The workspace and its bytes; without one, `need` bytes that belong to the stream the
    kernels run on, so that torch gives them to nobody else before those are done."""
    if workspace is None:
        if isinstance(stream, int):  # 1 is the legacy default stream, torch's 0
            stream = torch.cuda.ExternalStream(stream if stream != 1 else 0)
        with nullcontext() if stream is None else torch.cuda.stream(stream):
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


def _check(status: int):
    if status != NVFP4_OK:
        raise NVFP4Error(status, nvfp4_last_error())


def _in_dtype(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return NVFP4_IN_BF16
    if x.dtype == torch.float32:
        return NVFP4_IN_FP32
    raise TypeError(f"x must be bfloat16 or float32, got {x.dtype}")


def _matrix(x: torch.Tensor):
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D tensor")
    return x.shape[0], x.shape[1]


def nvfp4_last_error() -> str:
    return load_library().nvfp4_last_error().decode()


def nvfp4_amax(x: torch.Tensor, row_amax=None, col_amax=None, tensor_amax=None, noop=None,
               stream=None) -> None:
    rows, cols = _matrix(x)
    _check(load_library().nvfp4_amax(_ptr(x), _in_dtype(x), rows, cols, _ptr(row_amax),
                                     _ptr(col_amax), _ptr(tensor_amax), _ptr(noop),
                                     _stream(stream)))


def nvfp4_quantize_rowwise(x: torch.Tensor, cfg: Config, row: Out, noop=None, stream=None):
    rows, cols = _matrix(x)
    r = row._c()
    _check(load_library().nvfp4_quantize_rowwise(_ptr(x), _in_dtype(x), rows, cols,
                                                 C.byref(cfg), C.byref(r), _ptr(noop),
                                                 _stream(stream)))


def nvfp4_quantize_columnwise(x: torch.Tensor, cfg: Config, col: Out, noop=None, stream=None):
    rows, cols = _matrix(x)
    c = col._c()
    _check(load_library().nvfp4_quantize_columnwise(_ptr(x), _in_dtype(x), rows, cols,
                                                    C.byref(cfg), C.byref(c), _ptr(noop),
                                                    _stream(stream)))


def nvfp4_rht16(x: torch.Tensor, sign_mask: int, y: torch.Tensor, stream=None) -> None:
    """y (FP32, x's shape) = the random Hadamard transform of x along its rows, per
    column and per 16-row block, with the given 16-bit sign mask."""
    rows, cols = _matrix(x)
    if y.dtype != torch.float32 or tuple(y.shape) != (rows, cols) or not y.is_contiguous():
        raise ValueError("y must be a contiguous float32 tensor of x's shape")
    _check(load_library().nvfp4_rht16(_ptr(x), _in_dtype(x), rows, cols, sign_mask, _ptr(y),
                                      _stream(stream)))


def nvfp4_quantize_columnwise_rht(x: torch.Tensor, sign_mask: int, cfg: Config, col: Out,
                                  workspace: Optional[torch.Tensor] = None, noop=None,
                                  stream=None) -> None:
    """Columnwise quantization of the transformed x.  1x16 blocks: fused, no
    workspace.  16x16 blocks: workspace, a device buffer of at least 4 * rows * cols
    bytes, receives the transformed operand."""
    rows, cols = _matrix(x)
    c = col._c()
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().nvfp4_quantize_columnwise_rht(
        _ptr(x), _in_dtype(x), rows, cols, sign_mask, C.byref(cfg), C.byref(c), _ptr(workspace),
        nbytes, _ptr(noop), _stream(stream)))


def nvfp4_grouped_quantize_columnwise_rht(x: torch.Tensor, group_ends: torch.Tensor,
                                          sign_mask: int, cfg: Config, col: Out, noop=None,
                                          stream=None) -> None:
    """Grouped columnwise quantization of the transformed x (each group's amax)."""
    rows, cols = _matrix(x)
    c = col._c()
    _check(load_library().nvfp4_grouped_quantize_columnwise_rht(
        _ptr(x), _in_dtype(x), rows, cols, _ptr(group_ends), group_ends.numel(), sign_mask,
        C.byref(cfg), C.byref(c), _ptr(noop), _stream(stream)))


def nvfp4_quantize_both_rht(x: torch.Tensor, sign_mask: int, cfg: Config, row: Out, col: Out,
                            noop=None, stream=None) -> None:
    """Rowwise quantization of x and columnwise quantization of the transformed x in
    one encode pass (1x16 blocks)."""
    rows, cols = _matrix(x)
    r, c = row._c(), col._c()
    _check(load_library().nvfp4_quantize_both_rht(
        _ptr(x), _in_dtype(x), rows, cols, sign_mask, C.byref(cfg), C.byref(r), C.byref(c),
        _ptr(noop), _stream(stream)))


def nvfp4_quantize_both(x: torch.Tensor, cfg: Config, row: Out, col: Out, noop=None,
                        stream=None):
    rows, cols = _matrix(x)
    r, c = row._c(), col._c()
    _check(load_library().nvfp4_quantize_both(_ptr(x), _in_dtype(x), rows, cols, C.byref(cfg),
                                              C.byref(r), C.byref(c), _ptr(noop),
                                              _stream(stream)))


def nvfp4_dequantize(codes, scales, amax, mode: int, rows: int, cols: int, bound: float,
                     out: torch.Tensor, stream=None) -> None:
    if out.dtype == torch.bfloat16:
        od = NVFP4_OUT_BF16
    elif out.dtype == torch.float32:
        od = NVFP4_OUT_FP32
    else:
        raise TypeError("out must be bfloat16 or float32")
    _check(load_library().nvfp4_dequantize(_ptr(codes), _ptr(scales), _ptr(amax), mode, rows,
                                           cols, bound, _ptr(out), od, _stream(stream)))


def nvfp4_grouped_amax(x: torch.Tensor, group_ends: torch.Tensor, group_amax: torch.Tensor,
                       row_amax_expanded=None, noop=None, stream=None) -> None:
    rows, cols = _matrix(x)
    _check(load_library().nvfp4_grouped_amax(_ptr(x), _in_dtype(x), rows, cols,
                                             _ptr(group_ends), int(group_ends.numel()),
                                             _ptr(group_amax), _ptr(row_amax_expanded),
                                             _ptr(noop), _stream(stream)))


def nvfp4_grouped_quantize_rowwise(x: torch.Tensor, group_ends: torch.Tensor, cfg: Config,
                                   row: Out, group_amax=None, noop=None, stream=None) -> None:
    rows, cols = _matrix(x)
    r = row._c()
    _check(load_library().nvfp4_grouped_quantize_rowwise(
        _ptr(x), _in_dtype(x), rows, cols, _ptr(group_ends), int(group_ends.numel()),
        C.byref(cfg), C.byref(r), _ptr(group_amax), _ptr(noop), _stream(stream)))


def nvfp4_grouped_quantize_rowwise_padded(x: torch.Tensor, ragged_ends: torch.Tensor,
                                          padded_ends: torch.Tensor, padded_rows: int,
                                          cfg: Config, row: Out, group_amax: torch.Tensor,
                                          noop=None, stream=None) -> None:
    tokens, cols = _matrix(x)
    r = row._c()
    _check(load_library().nvfp4_grouped_quantize_rowwise_padded(
        _ptr(x), _in_dtype(x), tokens, cols, _ptr(ragged_ends), _ptr(padded_ends),
        int(ragged_ends.numel()), int(padded_rows), C.byref(cfg), C.byref(r), _ptr(group_amax),
        _ptr(noop), _stream(stream)))


def nvfp4_grouped_quantize_columnwise(x: torch.Tensor, group_ends: torch.Tensor, cfg: Config,
                                      col: Out, noop=None, stream=None) -> None:
    rows, cols = _matrix(x)
    c = col._c()
    _check(load_library().nvfp4_grouped_quantize_columnwise(
        _ptr(x), _in_dtype(x), rows, cols, _ptr(group_ends), int(group_ends.numel()),
        C.byref(cfg), C.byref(c), _ptr(noop), _stream(stream)))


def nvfp4_device_status(reset: bool = False, raise_on_timeout: bool = False) -> int:
    """The device status word's NVFP4_DEVICE_* bits.  The C call returns
    NVFP4_ERR_TIMEOUT when the timeout bit is set; that raises here only with
    raise_on_timeout, else the bits are returned as for any other state."""
    v = C.c_int32(0)
    rc = load_library().nvfp4_device_status(C.byref(v), int(reset))
    if rc != NVFP4_ERR_TIMEOUT or raise_on_timeout:
        _check(rc)
    return v.value


def nvfp4_selftest_scale_division(S: torch.Tensor, e_out: torch.Tensor, stream=None) -> None:
    """e_out[i, s8] = the encode kernels' fl(S[i] / decode(s8)) for s8 = 0 .. 126."""
    if S.dtype != torch.float32 or not S.is_contiguous():
        raise TypeError("S must be contiguous float32")
    if e_out.dtype != torch.float32 or e_out.numel() != S.numel() * 127:
        raise TypeError("e_out must be float32 with S.numel() * 127 elements")
    _check(load_library().nvfp4_selftest_scale_division(_ptr(S), S.numel(), _ptr(e_out),
                                                        _stream(stream)))


def nvfp4_selftest_wait_timeout(limit_ns: int, out: torch.Tensor, stream=None) -> None:
    """Run the bounded-wait self-test: a wait that nothing completes, given up after
    limit_ns nanoseconds (out: one device uint32, left untouched when it gives up)."""
    if out.dtype not in (torch.int32, torch.uint32) or out.numel() < 1:
        raise TypeError("out must hold at least one 32-bit integer")
    _check(load_library().nvfp4_selftest_wait_timeout(int(limit_ns), _ptr(out), _stream(stream)))


def nvfp4_selftest_convert(x: torch.Tensor, e2m1_out=None, e4m3_out=None, stream=None) -> None:
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise TypeError("x must be contiguous float32")
    _check(load_library().nvfp4_selftest_convert(_ptr(x), x.numel(), _ptr(e2m1_out),
                                                 _ptr(e4m3_out), _stream(stream)))


class _COperand(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("amax", C.c_void_p),
                ("mode", C.c_int32), ("bound", C.c_float)]


@dataclass
class Operand:
    """One nvfp4_gemm operand (nvfp4_operand): K-major codes [lines][k/2], scales
    [lines][k/16], amax [lines] (ROW_SCALED) or [1] (PER_TENSOR), the bound it was
    quantized with.  Out.as_operand() builds one from a quantize output."""
    codes: torch.Tensor
    scales: torch.Tensor
    amax: torch.Tensor
    mode: int
    bound: float

    def _c(self) -> _COperand:
        return _COperand(_ptr(self.codes), _ptr(self.scales), _ptr(self.amax), self.mode,
                         self.bound)


def nvfp4_gemm_workspace_size(m: int, n: int, k: int) -> int:
    v = C.c_uint64(0)
    _check(load_library().nvfp4_gemm_workspace_size(m, n, k, C.byref(v)))
    return v.value


def nvfp4_gemm(a: Operand, b: Operand, d: torch.Tensor, workspace: Optional[torch.Tensor] = None,
               stream=None) -> None:
    """d [m][n] (bfloat16 or float32) = dequant(a) x dequant(b)^T on the tensor cores.
    workspace: uint8 device tensor of nvfp4_gemm_workspace_size(m, n, k) bytes (allocated
    here with torch if not given)."""
    if d.dim() != 2 or not d.is_contiguous():
        raise ValueError("d must be a contiguous 2-D tensor")
    if d.dtype == torch.bfloat16:
        od = NVFP4_OUT_BF16
    elif d.dtype == torch.float32:
        od = NVFP4_OUT_FP32
    else:
        raise TypeError("d must be bfloat16 or float32")
    m, n = d.shape
    k = a.codes.shape[1] * 2
    if a.codes.shape[0] != m or b.codes.shape[0] != n or b.codes.shape[1] * 2 != k:
        raise ValueError("operand shapes do not match d")
    need = nvfp4_gemm_workspace_size(m, n, k)
    workspace, size = _workspace(workspace, need, d.device, stream)
    ca, cb = a._c(), b._c()
    _check(load_library().nvfp4_gemm(C.byref(ca), C.byref(cb), m, n, k, _ptr(d), od,
                                      _ptr(workspace), size, _stream(stream)))


def nvfp4_grouped_gemm_workspace_size(rows: int, n: int, k: int, num_groups: int) -> int:
    v = C.c_uint64(0)
    _check(load_library().nvfp4_grouped_gemm_workspace_size(rows, n, k, num_groups, C.byref(v)))
    return v.value


def nvfp4_grouped_gemm(a: Operand, b: Operand, group_ends: torch.Tensor, d: torch.Tensor,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """d [rows][n] = per group g: dequant(a rows of g) x dequant(b rows [g*n, (g+1)*n))^T.
    group_ends: device int64 [groups]; b.codes has groups * n rows."""
    if d.dim() != 2 or not d.is_contiguous():
        raise ValueError("d must be a contiguous 2-D tensor")
    if d.dtype == torch.bfloat16:
        od = NVFP4_OUT_BF16
    elif d.dtype == torch.float32:
        od = NVFP4_OUT_FP32
    else:
        raise TypeError("d must be bfloat16 or float32")
    rows, n = d.shape
    groups = int(group_ends.numel())
    k = a.codes.shape[1] * 2
    if a.codes.shape[0] != rows or b.codes.shape[0] != groups * n or b.codes.shape[1] * 2 != k:
        raise ValueError("operand shapes do not match d and the group count")
    need = nvfp4_grouped_gemm_workspace_size(rows, n, k, groups)
    workspace, size = _workspace(workspace, need, d.device, stream)
    ca, cb = a._c(), b._c()
    _check(load_library().nvfp4_grouped_gemm(C.byref(ca), C.byref(cb), _ptr(group_ends), groups,
                                              rows, n, k, _ptr(d), od, _ptr(workspace),
                                              size, _stream(stream)))


def nvfp4_grouped_gemm_wgrad(a: Operand, b: Operand, group_ends: torch.Tensor, d: torch.Tensor,
                             workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """d [groups][m][n]: per group g, dequant(a) x dequant(b)^T over g's token range of K.
    a [m][tokens/2], b [n][tokens/2] (columnwise outputs); group_ends device int64."""
    if d.dim() != 3 or not d.is_contiguous():
        raise ValueError("d must be a contiguous 3-D tensor [groups][m][n]")
    if d.dtype == torch.bfloat16:
        od = NVFP4_OUT_BF16
    elif d.dtype == torch.float32:
        od = NVFP4_OUT_FP32
    else:
        raise TypeError("d must be bfloat16 or float32")
    groups, m, n = d.shape
    tokens = a.codes.shape[1] * 2
    if (groups != group_ends.numel() or a.codes.shape[0] != m or b.codes.shape[0] != n
            or b.codes.shape[1] * 2 != tokens):
        raise ValueError("operand shapes do not match d and the group count")
    need = nvfp4_gemm_workspace_size(m, n, tokens)
    workspace, size = _workspace(workspace, need, d.device, stream)
    ca, cb = a._c(), b._c()
    _check(load_library().nvfp4_grouped_gemm_wgrad(C.byref(ca), C.byref(cb), _ptr(group_ends),
                                                    groups, m, n, tokens, _ptr(d), od,
                                                    _ptr(workspace), size,
                                                    _stream(stream)))


def nvfp4_gemm_static_ws(a: Operand, b: Operand, d: torch.Tensor, stream=None) -> None:
    """nvfp4_gemm with the library's static device workspace (no workspace argument)."""
    if d.dim() != 2 or not d.is_contiguous():
        raise ValueError("d must be a contiguous 2-D tensor")
    if d.dtype == torch.bfloat16:
        od = NVFP4_OUT_BF16
    elif d.dtype == torch.float32:
        od = NVFP4_OUT_FP32
    else:
        raise TypeError("d must be bfloat16 or float32")
    m, n = d.shape
    k = a.codes.shape[1] * 2
    if a.codes.shape[0] != m or b.codes.shape[0] != n or b.codes.shape[1] * 2 != k:
        raise ValueError("operand shapes do not match d")
    ca, cb = a._c(), b._c()
    _check(load_library().nvfp4_gemm_static_ws(C.byref(ca), C.byref(cb), m, n, k, _ptr(d), od,
                                                _stream(stream)))


# ---------------------------------------------------------------- layer operators


class _CFp8Out(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scale", C.c_void_p), ("block", C.c_int32)]


@dataclass
class Fp8Out:
    """An 8-bit rowwise output: E4M3 codes [rows][cols] (uint8 or float8_e4m3fn), FP32 scale
    [rows] (block 0) or [rows][ceil(cols/128)] (block 128)."""
    codes: torch.Tensor
    scale: torch.Tensor
    block: int = 0


class _CEpilogue(C.Structure):
    _fields_ = [("bias", C.c_void_p), ("bias_dtype", C.c_int32), ("act", C.c_int32),
                ("residual", C.c_void_p), ("z", C.c_void_p)]


class _CTensor(C.Structure):
    _fields_ = [("data", C.c_void_p), ("out", C.c_void_p), ("n", C.c_int64),
                ("dtype", C.c_int32)]


_DTYPE_CODES = {torch.bfloat16: NVFP4_IN_BF16, torch.float32: NVFP4_IN_FP32}


def _like(name: str, t: Optional[torch.Tensor], shape, dtype) -> Optional[int]:
    """The address of an optional contiguous tensor of the given shape and type."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _floats(name: str, t: Optional[torch.Tensor], n: int) -> Optional[int]:
    """The address of an optional FP32 vector of n elements (any contiguous shape)."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous float32 with {n} elements")
    return t.data_ptr()


def _on_gpu(*tensors) -> None:
    """Refuse a host tensor: the kernels would take its address for device memory."""
    for t in tensors:
        if t is not None and t.get_device() < 0:
            raise ValueError(f"every tensor must be on the GPU, got one on {t.device}")


def _operand_sizes(name: str, o: Operand, lines: int, k: int) -> None:
    """The kernels read codes [lines][k/2], scales [lines][k/16] and one or `lines` amax."""
    c, s, a = o.codes, o.scales, o.amax
    if not c.is_contiguous() or s.numel() != lines * (k // 16) or not s.is_contiguous() or \
            c.element_size() != 1 or s.element_size() != 1:
        raise ValueError(f"{name}: codes [lines][k/2] and scales [lines][k/16] must be contiguous "
                         "bytes")
    if a.dtype is not torch.float32 or not a.is_contiguous() or \
            a.numel() < (lines if o.mode == NVFP4_ROW_SCALED else 1):
        raise ValueError(f"{name}.amax must be contiguous float32, one per line or one")


def _vector(name: str, t: torch.Tensor, n: int) -> int:
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} elements")
    return _in_dtype(t)


def nvfp4_add_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float,
                      residual: Optional[torch.Tensor] = None,
                      h: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                      rstd: Optional[torch.Tensor] = None, fp8: Optional[Fp8Out] = None,
                      row: Optional[Out] = None, cfg: Optional[Config] = None,
                      stream=None) -> None:
    """h = x + residual, y = h * weight / sqrt(mean(h^2) + eps) of each row of x [rows][cols]
    (bfloat16 or float32).  Outputs: h, y (x's type), rstd [rows], and one quantized form of
    the FP32 y: fp8 (Fp8Out) or row with cfg (rowwise NVFP4, as nvfp4_quantize_rowwise)."""
    rows, cols = _matrix(x)
    shape, dtype = x.shape, x.dtype
    cfp8 = crow = None
    quantized = ()
    if fp8 is not None:
        if fp8.codes.shape != shape or not fp8.codes.is_contiguous() or \
                fp8.codes.element_size() != 1:
            raise ValueError("fp8.codes must be a contiguous one-byte tensor of x's shape")
        scale = _floats("fp8.scale", fp8.scale, rows * (-(-cols // 128) if fp8.block else 1))
        cfp8 = C.byref(_CFp8Out(fp8.codes.data_ptr(), scale, fp8.block))
        quantized = (fp8.codes, fp8.scale)
    if row is not None:
        if cfg is None:
            raise ValueError("a row output needs cfg")
        for name, t, n in (("codes", row.codes, rows * ((cols + 1) // 2)),
                           ("scales", row.scales, rows * ((cols + 15) // 16))):
            if t.element_size() != 1 or t.numel() != n or not t.is_contiguous():
                raise ValueError(f"row.{name} must be contiguous bytes, {n} of them")
        lines = rows if cfg.mode == NVFP4_ROW_SCALED else 1
        _floats("row.amax", row.amax, lines)
        _floats("row.amax_in", row.amax_in, lines)
        crow = C.byref(row._c())
        quantized += (row.codes, row.scales, row.amax, row.amax_in)
    args = (x.data_ptr(), _like("residual", residual, shape, dtype), _in_dtype(x),
            weight.data_ptr(), _vector("weight", weight, cols), rows, cols, eps,
            _like("h", h, shape, dtype), _like("y", y, shape, dtype), _floats("rstd", rstd, rows),
            cfp8, C.byref(cfg) if cfg is not None else None, crow)
    _on_gpu(x, weight, residual, h, y, rstd, *quantized)
    _check(load_library().nvfp4_add_rmsnorm(*args, _stream(stream)))


def nvfp4_add_rmsnorm_backward_workspace_size(rows: int, cols: int) -> int:
    v = C.c_uint64(0)
    _check(load_library().nvfp4_add_rmsnorm_backward_workspace_size(rows, cols, C.byref(v)))
    return v.value


def nvfp4_add_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                               rstd: torch.Tensor, dx: torch.Tensor,
                               dweight: Optional[torch.Tensor] = None,
                               dh: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of nvfp4_add_rmsnorm: dx (of x and of residual; dh, the gradient reaching h
    beside the norm's, is added) and dweight [cols] float32."""
    rows, cols = _matrix(h)
    shape, dtype = h.shape, h.dtype
    args = (_like("dy", dy, shape, dtype), h.data_ptr(), _like("dh", dh, shape, dtype),
            _in_dtype(h), weight.data_ptr(), _vector("weight", weight, cols),
            _floats("rstd", rstd, rows), rows, cols, _like("dx", dx, shape, dtype),
            _floats("dweight", dweight, cols))
    _on_gpu(dy, h, weight, rstd, dx, dweight, dh, workspace)
    size = 0
    if dweight is not None:
        need = 0 if workspace is not None else \
            nvfp4_add_rmsnorm_backward_workspace_size(rows, cols)
        workspace, size = _workspace(workspace, need, h.device, stream)
    _check(load_library().nvfp4_add_rmsnorm_backward(*args, _ptr(workspace), size,
                                                     _stream(stream)))


def nvfp4_gemm_bias_act_workspace_size(m: int, n: int, k: int) -> int:
    v = C.c_uint64(0)
    _check(load_library().nvfp4_gemm_bias_act_workspace_size(m, n, k, C.byref(v)))
    return v.value


def nvfp4_gemm_bias_act(a: Operand, b: Operand, d: torch.Tensor,
                        bias: Optional[torch.Tensor] = None, act: int = NVFP4_ACT_NONE,
                        residual: Optional[torch.Tensor] = None,
                        z: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """d [m][n] (bfloat16 or float32) = act(z) + residual, z = dequant(a) x dequant(b)^T +
    bias.  bias [n] bfloat16 or float32; residual and z (receives the pre-activation) have
    d's shape and type; residual may be d."""
    m, n = _matrix(d)
    od = NVFP4_OUT_FP32 if d.dtype == torch.float32 else NVFP4_OUT_BF16
    _in_dtype(d)
    k = a.codes.shape[1] * 2
    if a.codes.shape[0] != m or b.codes.shape[0] != n or b.codes.shape[1] * 2 != k:
        raise ValueError("operand shapes do not match d")
    shape, dtype = d.shape, d.dtype
    _operand_sizes("a", a, m, k)
    _operand_sizes("b", b, n, k)
    bd = _vector("bias", bias, n) if bias is not None else NVFP4_IN_FP32
    epi = _CEpilogue(_ptr(bias), bd, act, _like("residual", residual, shape, dtype),
                     _like("z", z, shape, dtype))
    _on_gpu(a.codes, a.scales, a.amax, b.codes, b.scales, b.amax, d, bias, residual, z, workspace)
    need = 0 if workspace is not None else nvfp4_gemm_bias_act_workspace_size(m, n, k)
    workspace, size = _workspace(workspace, need, d.device, stream)
    ca, cb = a._c(), b._c()
    _check(load_library().nvfp4_gemm_bias_act(C.byref(ca), C.byref(cb), m, n, k, C.byref(epi),
                                              _ptr(d), od, _ptr(workspace), size,
                                              _stream(stream)))


def nvfp4_bias_act_backward_workspace_size(rows: int, cols: int) -> int:
    v = C.c_uint64(0)
    _check(load_library().nvfp4_bias_act_backward_workspace_size(rows, cols, C.byref(v)))
    return v.value


def nvfp4_bias_act_backward(dd: torch.Tensor, z: Optional[torch.Tensor], act: int,
                            dz: torch.Tensor, dbias: Optional[torch.Tensor] = None,
                            row_amax: Optional[torch.Tensor] = None,
                            col_amax: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """dz = dd * act'(z), dbias [cols] = its column sums, row_amax [rows] / col_amax [cols] =
    the maxima of |dz|, ready to be the amax_in of the quantization of dz."""
    rows, cols = _matrix(dd)
    shape, dtype = dd.shape, dd.dtype
    args = (dd.data_ptr(), _like("z", z, shape, dtype), _in_dtype(dd), act, rows, cols,
            _like("dz", dz, shape, dtype), _floats("dbias", dbias, cols),
            _floats("row_amax", row_amax, rows), _floats("col_amax", col_amax, cols))
    _on_gpu(dd, z, dz, dbias, row_amax, col_amax, workspace)
    size = 0
    if dbias is not None or row_amax is not None or col_amax is not None:
        need = 0 if workspace is not None else nvfp4_bias_act_backward_workspace_size(rows, cols)
        workspace, size = _workspace(workspace, need, dd.device, stream)
    _check(load_library().nvfp4_bias_act_backward(*args, _ptr(workspace), size, _stream(stream)))


def nvfp4_clip_grad_norm_workspace_size() -> int:
    v = C.c_uint64(0)
    _check(load_library().nvfp4_clip_grad_norm_workspace_size(C.byref(v)))
    return v.value


def _tensor_list(tensors, out):
    """The tensors as an array of nvfp4_tensor: four 64-bit words each (data, out, n, and
    dtype with its padding)."""
    T = torch.Tensor
    data, sizes = list(map(T.data_ptr, tensors)), list(map(T.numel, tensors))
    types = [t.dtype for t in tensors]
    if not all(map(T.is_contiguous, tensors)):
        raise ValueError("every tensor must be contiguous")
    codes = [_DTYPE_CODES.get(t, -1) for t in types]
    if -1 in codes:
        raise TypeError(f"tensors must be bfloat16 or float32, got {types[codes.index(-1)]}")
    to = data
    if out is not None:
        if [o.dtype for o in out] != types or list(map(T.numel, out)) != sizes or \
                not all(map(T.is_contiguous, out)):
            raise ValueError("out must be contiguous tensors of the tensors' types and sizes")
        to = list(map(T.data_ptr, out))
    if -1 in map(T.get_device, tensors) or out is not None and -1 in map(T.get_device, out):
        _on_gpu(*tensors, *(out or ()))
    words = [0] * (4 * len(data))
    words[0::4], words[1::4], words[2::4], words[3::4] = data, to, sizes, codes
    return array("q", words)


def nvfp4_grad_norm(tensors, norm: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """norm [1] (float32) = the 2-norm of all tensors (bfloat16 or float32) together."""
    _floats("norm", norm, 1)
    items = _tensor_list(tensors, None)
    _on_gpu(norm, workspace)
    need = 0 if workspace is not None else nvfp4_clip_grad_norm_workspace_size()
    workspace, size = _workspace(workspace, need, norm.device, stream)
    _check(load_library().nvfp4_grad_norm(items.buffer_info()[0], len(tensors), _ptr(norm),
                                          _ptr(workspace), size,
                                          _stream(stream)))


def nvfp4_clip_grad_norm(tensors, max_norm: float, norm: torch.Tensor, out=None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Scale the tensors (in place, or into the list out) by min(1, max_norm / (norm + 1e-6));
    norm [1] (float32) receives their global 2-norm before that."""
    _floats("norm", norm, 1)
    if out is not None and len(out) != len(tensors):
        raise ValueError("out must have one tensor for each tensor")
    items = _tensor_list(tensors, out)
    _on_gpu(norm, workspace)
    need = 0 if workspace is not None else nvfp4_clip_grad_norm_workspace_size()
    workspace, size = _workspace(workspace, need, norm.device, stream)
    _check(load_library().nvfp4_clip_grad_norm(items.buffer_info()[0], len(tensors), max_norm,
                                               _ptr(norm), _ptr(workspace), size,
                                               _stream(stream)))


def alloc_out(lines: int, n: int, amax_len: int, device="cuda", fill=None) -> Out:
    """Allocate one output direction with torch (codes, scales, amax)."""
    codes = torch.empty(lines, (n + 1) // 2, dtype=torch.uint8, device=device)
    scales = torch.empty(lines, (n + 15) // 16, dtype=torch.uint8, device=device)
    amax = torch.empty(amax_len, dtype=torch.float32, device=device)
    if fill is not None:
        codes.fill_(fill)
        scales.fill_(fill)
    return Out(codes, scales, amax)
