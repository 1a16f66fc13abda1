"""Python binding of libhgemm.so, the GB300 FP16 tensor-core GEMM C = A·B.

Argument marshalling only: every step of the product runs in the library's
CUDA kernels (see ``include/hgemm.h`` for the contract). Functions carry the
C names. Matrices may be given as torch tensors (their ``data_ptr()`` is
passed), numpy arrays (host memory, for ``hgemm_host``) or raw integer
addresses. Streams may be a ``torch.cuda.Stream``, a raw handle, or None for
torch's current stream.

Layouts, as in "Nvidia Tensor Core-MMA PTX编程入门", §4 示例: A is M×K
row-major, B is K×N column-major (pass it as an (N, K) row-major array whose
row j is column j of B), C is M×N row-major; all FP16.

If the shared library has not been built, every call raises: there is no
fallback implementation.
"""

from __future__ import annotations

import ctypes
import os

__all__ = [
    "HGEMM_OK", "HGEMM_ERR_INVALID_ARG", "HGEMM_ERR_ALIAS", "HGEMM_ERR_UNSUPPORTED_DEVICE",
    "HGEMM_ERR_CUDA", "HGEMM_ERR_TIMEOUT", "HGEMM_ERR_DEBUG_CHECK", "hgemm_debug_build", "hgemm_debug_code",
    "hgemm_debug_selftest", "HGEMM_PATH_NONE", "HGEMM_PATH_ZERO",
    "HGEMM_PATH_TC", "HGEMM_PATH_SKINNY", "HGEMM_PATH_GENERIC", "HGEMM_PATH_TC_PAIR",
    "HGEMM_PATH_TC_WIDE", "HGEMM_PATH_TC_NARROW", "HGEMM_MAX_DIM",
    "HgemmError", "library_path", "load", "hgemm", "hgemm_host", "hgemm_select_path",
    "hgemm_force_path", "hgemm_device_status", "hgemm_last_cuda_error",
    "hgemm_status_string", "hgemm_version", "hgemm_set_wait_timeout", "hgemm_debug_inject",
    "hgemm_force_split", "hgemm_launch_floor", "hgemm_ex", "hgemm_strided", "hgemm_trmm", "hgemm_trsm", "hgemm_trsm_ws", "hgemm_trsm_workspace_size", "hgemm_trsm_noalloc", "hgemm_trsm_op", "HGEMM_OP_N", "HGEMM_OP_T", "hgemm_layout", "HGEMM_TRMM_MAX_N", "HGEMM_TRSM_NOALLOC_MAX_BYTES",
    "hgemm_force_trsm_schedule", "hgemm_trsm_last_schedule", "HGEMM_TRSM_AUTO", "HGEMM_TRSM_SUBSTITUTION",
    "HGEMM_TRSM_RECURSIVE", "HGEMM_TRSM_CHAIN", "HGEMM_TRSM_CHAIN_FUSED", "HGEMM_TRSM_CHAIN_SPLIT",
    "HGEMM_A_ROW_MAJOR", "HGEMM_A_COL_MAJOR", "HGEMM_B_COL_MAJOR", "HGEMM_B_ROW_MAJOR",
    "HGEMM_INJECT_NONE", "HGEMM_INJECT_DROP_ARRIVAL", "matmul",
    "hgemm_linear", "hgemm_linear_dgrad", "hgemm_linear_wgrad", "hgemm_layernorm_forward",
    "hgemm_layernorm_backward", "hgemm_layernorm_backward_workspace_size", "hgemm_ckpt8_save", "hgemm_ckpt8_load",
    "HGEMM_ACT_NONE", "HGEMM_ACT_RELU", "HGEMM_ACT_GELU", "HGEMM_ACT_SILU", "HGEMM_ACT_GELU_ERF",
    "HGEMM_CKPT8_GROUP",
    "hgemm_residual_norm_forward", "hgemm_residual_norm_backward", "hgemm_residual_norm_backward_workspace_size",
    "HGEMM_NORM_NONE", "HGEMM_NORM_LAYER", "HGEMM_NORM_RMS",
    "hgemm_adamw", "hgemm_adamw_rounded", "hgemm_adamw_check", "hgemm_adamw_tensors", "hgemm_adamw_dynamic", "hgemm_adamw_load", "AdamwTensors", "HGEMM_TYPE_F16",
    "HGEMM_TYPE_F32", "HGEMM_ROUND_NEAREST", "HGEMM_ROUND_RANDOM", "hgemm_experts", "hgemm_experts_workspace_size", "HGEMM_EXPERTS_MAX_TOKENS",
    "HGEMM_EXPERTS_MAX_CHOICES", "HGEMM_EXPERTS_MAX", "HGEMM_EXPERTS_MAX_WIDTH",
]

HGEMM_OK = 0
HGEMM_ERR_INVALID_ARG = -1
HGEMM_ERR_ALIAS = -2
HGEMM_ERR_UNSUPPORTED_DEVICE = -3
HGEMM_ERR_CUDA = -4
HGEMM_ERR_TIMEOUT = -5
HGEMM_ERR_DEBUG_CHECK = -6
HGEMM_TRMM_MAX_N = 16384
HGEMM_TRSM_NOALLOC_MAX_BYTES = (17 << 19) + 4096
HGEMM_TRSM_AUTO = 0
HGEMM_TRSM_SUBSTITUTION = 1
HGEMM_TRSM_RECURSIVE = 2
HGEMM_TRSM_CHAIN = 3
HGEMM_TRSM_CHAIN_FUSED = 4
HGEMM_TRSM_CHAIN_SPLIT = 5
HGEMM_OP_N = 0
HGEMM_OP_T = 1
HGEMM_A_ROW_MAJOR = 0
HGEMM_A_COL_MAJOR = 1
HGEMM_B_COL_MAJOR = 0
HGEMM_B_ROW_MAJOR = 1

HGEMM_ACT_NONE = 0
HGEMM_ACT_RELU = 1
HGEMM_ACT_GELU = 2
HGEMM_ACT_SILU = 3
HGEMM_ACT_GELU_ERF = 4
HGEMM_CKPT8_GROUP = 64

HGEMM_NORM_NONE = 0
HGEMM_NORM_LAYER = 1
HGEMM_NORM_RMS = 2

HGEMM_TYPE_F16 = 0
HGEMM_TYPE_F32 = 1

HGEMM_ROUND_NEAREST = 0
HGEMM_ROUND_RANDOM = 1

HGEMM_EXPERTS_MAX_TOKENS = 64
HGEMM_EXPERTS_MAX_CHOICES = 16
HGEMM_EXPERTS_MAX = 512
HGEMM_EXPERTS_MAX_WIDTH = 1 << 20

HGEMM_PATH_NONE = 0
HGEMM_PATH_ZERO = 1
HGEMM_PATH_TC = 2
HGEMM_PATH_SKINNY = 3
HGEMM_PATH_GENERIC = 4
HGEMM_PATH_TC_PAIR = 5
HGEMM_PATH_TC_WIDE = 6
HGEMM_PATH_TC_NARROW = 7

HGEMM_MAX_DIM = 0x7FFFFFFF

HGEMM_INJECT_NONE = 0
HGEMM_INJECT_DROP_ARRIVAL = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
# HGEMM_LIBRARY_VARIANT=debug: the -DHGEMM_DEBUG build with device-side checks
_LIB_PATH = (os.path.join(_HERE, "_build", "debug", "libhgemm.so")
             if os.environ.get("HGEMM_LIBRARY_VARIANT") == "debug"
             else os.path.join(_HERE, "_build", "libhgemm.so"))
_lib = None


class HgemmError(RuntimeError):
    """A negative status from libhgemm."""

    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {hgemm_status_string(status)} (status {status})"
        if status == HGEMM_ERR_CUDA:
            msg += f", cudaError {hgemm_last_cuda_error()}"
        super().__init__(msg)


def library_path() -> str:
    return _LIB_PATH


def load():
    """Loads libhgemm.so (built by tensor_core_dense_fp16_gb300.build.build())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"{_LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc)")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.hgemm.argtypes = [vp, vp, vp, i64, i64, i64, vp]
    lib.hgemm.restype = i32
    lib.hgemm_ex.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.c_float, ctypes.c_float, vp,
                             i32, vp]
    lib.hgemm_ex.restype = i32
    lib.hgemm_strided.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, i64, ctypes.c_float,
                                  ctypes.c_float, vp, i32, vp]
    lib.hgemm_strided.restype = i32
    lib.hgemm_trmm.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, ctypes.c_float, vp]
    lib.hgemm_trmm.restype = i32
    lib.hgemm_trsm.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, ctypes.c_float, vp]
    lib.hgemm_trsm.restype = i32
    lib.hgemm_trsm_ws.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, ctypes.c_float, vp, ctypes.c_size_t, vp]
    lib.hgemm_trsm_ws.restype = i32
    lib.hgemm_trsm_workspace_size.argtypes = [i64]
    lib.hgemm_trsm_workspace_size.restype = ctypes.c_size_t
    lib.hgemm_trsm_op.argtypes = [i32, vp, i64, vp, i64, vp, i64, i64, i64, ctypes.c_float, vp,
                                  ctypes.c_size_t, vp]
    lib.hgemm_trsm_op.restype = i32
    lib.hgemm_trsm_noalloc.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, ctypes.c_float, vp]
    lib.hgemm_trsm_noalloc.restype = i32
    lib.hgemm_layout.argtypes = [i32, i32, vp, i64, vp, i64, vp, i64, i64, i64, i64, ctypes.c_float,
                                 ctypes.c_float, vp, i32, vp]
    lib.hgemm_layout.restype = i32
    lib.hgemm_host.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp, vp]
    lib.hgemm_host.restype = i32
    lib.hgemm_select_path.argtypes = [vp, vp, vp, i64, i64, i64]
    lib.hgemm_select_path.restype = i32
    lib.hgemm_force_path.argtypes = [i32]
    lib.hgemm_force_path.restype = i32
    lib.hgemm_device_status.argtypes = [vp]
    lib.hgemm_device_status.restype = i32
    lib.hgemm_last_cuda_error.argtypes = []
    lib.hgemm_last_cuda_error.restype = i32
    lib.hgemm_status_string.argtypes = [i32]
    lib.hgemm_status_string.restype = ctypes.c_char_p
    lib.hgemm_version.argtypes = []
    lib.hgemm_version.restype = i32
    lib.hgemm_set_wait_timeout.argtypes = [ctypes.c_ulonglong]
    lib.hgemm_set_wait_timeout.restype = i32
    lib.hgemm_debug_inject.argtypes = [i32]
    lib.hgemm_debug_inject.restype = i32
    lib.hgemm_force_split.argtypes = [i32, i32]
    lib.hgemm_force_split.restype = i32
    lib.hgemm_launch_floor.argtypes = [i32, vp]
    lib.hgemm_launch_floor.restype = i32
    lib.hgemm_force_trsm_schedule.argtypes = [i32]
    lib.hgemm_force_trsm_schedule.restype = i32
    f32 = ctypes.c_float
    lib.hgemm_linear.argtypes = [vp, i64, vp, i64, vp, i32, vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64, vp]
    lib.hgemm_linear_dgrad.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, i32, vp, i64, vp, i64, i64, i64, i64, vp]
    lib.hgemm_linear_wgrad.argtypes = [vp, i64, vp, i64, vp, i64, vp, i32, i64, i64, i64, vp]
    lib.hgemm_layernorm_forward.argtypes = [vp, i64, vp, vp, f32, vp, i64, vp, vp, i64, i64, vp]
    lib.hgemm_layernorm_backward.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp,
                                             ctypes.c_size_t, i64, i64, vp]
    lib.hgemm_ckpt8_save.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, vp]
    lib.hgemm_ckpt8_load.argtypes = [vp, i64, vp, i64, i32, vp, i64, i64, i64, vp]
    for name in ("hgemm_linear", "hgemm_linear_dgrad", "hgemm_linear_wgrad", "hgemm_layernorm_forward",
                 "hgemm_layernorm_backward", "hgemm_ckpt8_save", "hgemm_ckpt8_load"):
        getattr(lib, name).restype = i32
    lib.hgemm_layernorm_backward_workspace_size.argtypes = [i64, i64]
    lib.hgemm_layernorm_backward_workspace_size.restype = ctypes.c_size_t
    f64, size = ctypes.c_double, ctypes.c_size_t
    lib.hgemm_residual_norm_forward.argtypes = [vp, i64, f32, vp, i64, vp, i32, vp, vp, i32, vp, vp, f32, vp, i64, vp,
                                                i64, vp, i64, i64, vp]
    lib.hgemm_residual_norm_backward.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, f32, vp, i32, vp, vp, i32, vp, vp,
                                                 vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, size, i64, i64, vp]
    lib.hgemm_adamw.argtypes = [vp, i64, f64, f64, f64, f64, i64, f64, vp, vp]
    lib.hgemm_adamw_rounded.argtypes = [vp, i64, f64, f64, f64, f64, i64, f64, i32, vp, vp]
    lib.hgemm_adamw_check.argtypes = [vp, i64]
    lib.hgemm_adamw_load.argtypes = [vp, vp, vp, vp, vp, vp, i64, vp]
    lib.hgemm_experts.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, i64, vp, i32, i32, i64, i32, vp, i64, vp, i64, vp,
                                  vp, vp, size, i64, i64, i64, i64, vp]
    for name in ("hgemm_residual_norm_forward", "hgemm_residual_norm_backward", "hgemm_adamw", "hgemm_adamw_rounded",
                 "hgemm_adamw_check", "hgemm_adamw_load", "hgemm_experts"):
        getattr(lib, name).restype = i32
    lib.hgemm_residual_norm_backward_workspace_size.argtypes = [i64, i64]
    lib.hgemm_residual_norm_backward_workspace_size.restype = size
    lib.hgemm_experts_workspace_size.argtypes = [i64, i64, i64, i64, i64]
    lib.hgemm_experts_workspace_size.restype = size
    for name in ("hgemm_debug_build", "hgemm_debug_code", "hgemm_debug_selftest", "hgemm_trsm_last_schedule"):
        getattr(lib, name).argtypes = []
        getattr(lib, name).restype = i32
    _lib = lib
    return lib


# ----------------------------------------------------------------- marshalling

def _ptr(x) -> int | None:
    """Address of a torch tensor, numpy array, ctypes object or integer."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):          # torch.Tensor
        return int(x.data_ptr())
    if hasattr(x, "ctypes"):            # numpy.ndarray
        return int(x.ctypes.data)
    if isinstance(x, ctypes.c_void_p):
        return x.value
    raise TypeError(f"cannot take the address of {type(x).__name__}")


def _check_tensor(x, name: str, on_device: bool | None):
    """dtype and contiguity checks for torch tensors and numpy arrays."""
    if hasattr(x, "data_ptr") and hasattr(x, "dtype"):
        import torch
        if x.dtype != torch.float16:
            raise TypeError(f"{name} must be torch.float16, got {x.dtype}")
        if not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if on_device is True and not x.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if on_device is False and x.is_cuda:
            raise ValueError(f"{name} must be a host tensor")
    elif hasattr(x, "ctypes") and hasattr(x, "dtype"):
        import numpy as np
        if x.dtype != np.float16:
            raise TypeError(f"{name} must be float16, got {x.dtype}")
        if not x.flags["C_CONTIGUOUS"]:
            raise ValueError(f"{name} must be C-contiguous")
        if on_device is True:
            raise ValueError(f"{name} must be device memory, got a numpy array")


_torch = None              # torch, once a call has needed it
_raw_current_stream = None  # device index -> handle of torch's current stream


def _import_torch():
    global _torch, _raw_current_stream
    import torch
    torch.cuda.current_stream()  # initialises CUDA
    # the handle alone: torch.cuda.current_stream() makes a Stream object, 2.8 us against 0.1
    _raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _torch = torch
    return torch


def _stream(stream) -> int:
    if stream is None:
        torch = _torch or _import_torch()
        return int(_raw_current_stream(torch.cuda.current_device()))
    if isinstance(stream, int):
        return stream
    if hasattr(stream, "cuda_stream"):
        return int(stream.cuda_stream)
    raise TypeError(f"cannot use {type(stream).__name__} as a CUDA stream")


def _raise_on(status: int, where: str) -> int:
    if status < 0:
        raise HgemmError(status, where)
    return status


# --------------------------------------------------------------------- the ABI

def hgemm(A, B, C, M: int, N: int, K: int, stream=None) -> None:
    """C = A·B on `stream` (enqueued; synchronise the stream to read C)."""
    for x, n in ((A, "A"), (B, "B"), (C, "C")):
        _check_tensor(x, n, True)
    _raise_on(load().hgemm(_ptr(A), _ptr(B), _ptr(C), M, N, K, _stream(stream)), "hgemm")


def hgemm_ex(A, B, C, M: int, N: int, K: int, alpha: float = 1.0, beta: float = 0.0, bias=None,
             relu: bool = False, stream=None) -> None:
    """C = f(alpha·A·B + beta·C + bias[j]) on `stream`, f = ReLU if relu (see hgemm.h)."""
    for x, n in ((A, "A"), (B, "B"), (C, "C")):
        _check_tensor(x, n, True)
    if bias is not None:
        _check_tensor(bias, "bias", True)
    _raise_on(load().hgemm_ex(_ptr(A), _ptr(B), _ptr(C), M, N, K, float(alpha), float(beta),
                              _ptr(bias), int(bool(relu)), _stream(stream)), "hgemm_ex")


def hgemm_strided(A, lda: int, B, ldb: int, C, ldc: int, M: int, N: int, K: int,
                  alpha: float = 1.0, beta: float = 0.0, bias=None, relu: bool = False,
                  stream=None) -> None:
    """hgemm_ex on sub-matrices with row pitches (see hgemm.h). A, B, C may be
    tensors (their base address is used) or raw integer addresses."""
    _raise_on(load().hgemm_strided(_ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, M, N, K, float(alpha),
                                   float(beta), _ptr(bias), int(bool(relu)), _stream(stream)),
              "hgemm_strided")


def hgemm_layout(a_layout: int, b_layout: int, A, lda: int, B, ldb: int, C, ldc: int, M: int,
                 N: int, K: int, alpha: float = 1.0, beta: float = 0.0, bias=None,
                 relu: bool = False, stream=None) -> None:
    """hgemm_strided with a storage order per operand (HGEMM_A_* / HGEMM_B_*; see hgemm.h)."""
    _raise_on(load().hgemm_layout(int(a_layout), int(b_layout), _ptr(A), lda, _ptr(B), ldb, _ptr(C),
                                  ldc, M, N, K, float(alpha), float(beta), _ptr(bias),
                                  int(bool(relu)), _stream(stream)), "hgemm_layout")


def hgemm_trmm(A, lda: int, B, ldb: int, C, ldc: int, n: int, m: int, alpha: float = 1.0,
               stream=None) -> None:
    """C = alpha·Aᵀ·B, A lower triangular; column-major operands (see hgemm.h)."""
    _raise_on(load().hgemm_trmm(_ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, n, m, float(alpha),
                                _stream(stream)), "hgemm_trmm")


def hgemm_trsm(A, lda: int, B, ldb: int, X, ldx: int, n: int, m: int, alpha: float = 1.0,
               stream=None) -> None:
    """Solves Aᵀ·X = alpha·B for X, A lower triangular; column-major operands;
    X may be B itself (same pitch) to solve in place (see hgemm.h)."""
    _raise_on(load().hgemm_trsm(_ptr(A), lda, _ptr(B), ldb, _ptr(X), ldx, n, m, float(alpha),
                                _stream(stream)), "hgemm_trsm")


def hgemm_trsm_noalloc(A, lda: int, B, ldb: int, X, ldx: int, n: int, m: int, alpha: float = 1.0,
                       stream=None) -> None:
    """hgemm_trsm_ws with the library's fixed device workspace instead of one
    from the caller: allocates nothing (for callers that cannot allocate);
    n up to 8192 (see hgemm.h for the set-up on first use and the sharing
    of the workspace between calls)."""
    _raise_on(load().hgemm_trsm_noalloc(_ptr(A), lda, _ptr(B), ldb, _ptr(X), ldx, n, m, float(alpha),
                                        _stream(stream)), "hgemm_trsm_noalloc")


def hgemm_trsm_workspace_size(n: int) -> int:
    """Bytes of device workspace hgemm_trsm_ws uses for a triangle of order n."""
    return int(load().hgemm_trsm_workspace_size(n))


def hgemm_trsm_ws(A, lda: int, B, ldb: int, X, ldx: int, n: int, m: int, alpha: float = 1.0,
                  workspace=None, workspace_bytes: int | None = None, stream=None) -> None:
    """hgemm_trsm with a caller-owned device workspace (a tensor or an
    address; its size defaults to the tensor's bytes), see hgemm.h."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    _raise_on(load().hgemm_trsm_ws(_ptr(A), lda, _ptr(B), ldb, _ptr(X), ldx, n, m, float(alpha),
                                   _ptr(workspace), int(workspace_bytes), _stream(stream)), "hgemm_trsm_ws")


def hgemm_trsm_op(op: int, A, lda: int, B, ldb: int, X, ldx: int, n: int, m: int, alpha: float = 1.0,
                  workspace=None, workspace_bytes: int | None = None, stream=None) -> None:
    """Solves A·X = alpha·B (op = HGEMM_OP_N, the page's literal X = A\\B) or
    Aᵀ·X = alpha·B (HGEMM_OP_T) for X, A lower triangular, column-major
    operands; with an optional workspace as hgemm_trsm_ws takes (see hgemm.h)."""
    if workspace_bytes is None:
        workspace_bytes = (workspace.numel() * workspace.element_size() if hasattr(workspace, "numel")
                           else 0)
    _raise_on(load().hgemm_trsm_op(int(op), _ptr(A), lda, _ptr(B), ldb, _ptr(X), ldx, n, m, float(alpha),
                                   _ptr(workspace), int(workspace_bytes), _stream(stream)), "hgemm_trsm_op")


def hgemm_host(hA, hB, hC, M: int, N: int, K: int, dA, dB, dC, stream=None) -> None:
    """Host operands: H2D copies, the product and the D2H copy, all on `stream`."""
    for x, n in ((hA, "hA"), (hB, "hB"), (hC, "hC")):
        _check_tensor(x, n, False)
    for x, n in ((dA, "dA"), (dB, "dB"), (dC, "dC")):
        _check_tensor(x, n, True)
    _raise_on(load().hgemm_host(_ptr(hA), _ptr(hB), _ptr(hC), M, N, K, _ptr(dA), _ptr(dB),
                                _ptr(dC), _stream(stream)), "hgemm_host")


def hgemm_select_path(A, B, C, M: int, N: int, K: int) -> int:
    """The HGEMM_PATH_* hgemm would take (host logic only; raises on bad args)."""
    return _raise_on(load().hgemm_select_path(_ptr(A), _ptr(B), _ptr(C), M, N, K),
                     "hgemm_select_path")


def hgemm_force_path(path: int) -> None:
    _raise_on(load().hgemm_force_path(path), "hgemm_force_path")


def hgemm_force_trsm_schedule(schedule: int) -> None:
    """Testing aid: HGEMM_TRSM_RECURSIVE keeps solves with a workspace on the
    recursion's launches; HGEMM_TRSM_CHAIN (either plan), HGEMM_TRSM_CHAIN_FUSED
    or HGEMM_TRSM_CHAIN_SPLIT force the one persistent launch; HGEMM_TRSM_AUTO
    chooses."""
    _raise_on(load().hgemm_force_trsm_schedule(schedule), "hgemm_force_trsm_schedule")


def hgemm_trsm_last_schedule() -> int:
    """The HGEMM_TRSM_* schedule of the last solve enqueued on this thread."""
    return int(load().hgemm_trsm_last_schedule())


def hgemm_device_status(stream=None) -> int:
    """Synchronises `stream`; returns HGEMM_OK, HGEMM_ERR_TIMEOUT or (debug
    build) HGEMM_ERR_DEBUG_CHECK; raises otherwise."""
    st = load().hgemm_device_status(_stream(stream))
    if st in (HGEMM_OK, HGEMM_ERR_TIMEOUT, HGEMM_ERR_DEBUG_CHECK):
        return st
    raise HgemmError(st, "hgemm_device_status")


def hgemm_debug_build() -> int:
    return int(load().hgemm_debug_build())


def hgemm_debug_code() -> int:
    return int(load().hgemm_debug_code())


def hgemm_debug_selftest() -> int:
    return int(load().hgemm_debug_selftest())


def hgemm_launch_floor(pair_config: bool = True, stream=None) -> None:
    """Enqueues a kernel that does nothing (the pair kernel's launch
    configuration when pair_config), to time the fixed cost of a launch."""
    _raise_on(load().hgemm_launch_floor(1 if pair_config else 0, _stream(stream)), "hgemm_launch_floor")


def hgemm_last_cuda_error() -> int:
    return int(load().hgemm_last_cuda_error())


def hgemm_status_string(status: int) -> str:
    return load().hgemm_status_string(status).decode()


def hgemm_version() -> tuple[int, int]:
    v = int(load().hgemm_version())
    return v >> 16, v & 0xFFFF


def hgemm_set_wait_timeout(ns: int) -> None:
    """Time limit of every in-kernel wait for later calls (0: default 2 s)."""
    _raise_on(load().hgemm_set_wait_timeout(int(ns)), "hgemm_set_wait_timeout")


def hgemm_debug_inject(what: int) -> None:
    """Testing aid for the watchdog (HGEMM_INJECT_*); see include/hgemm.h."""
    _raise_on(load().hgemm_debug_inject(int(what)), "hgemm_debug_inject")


def hgemm_force_split(split: int, tile_n: int) -> None:
    """Testing aid: the split-K configuration for later calls ((0, 0): automatic)."""
    _raise_on(load().hgemm_force_split(int(split), int(tile_n)), "hgemm_force_split")


def matmul(a, b_cols, out=None, stream=None):
    """Convenience: a (M, K) and b_cols (N, K) CUDA float16 tensors -> (M, N).

    Row j of ``b_cols`` is column j of B. Allocates ``out`` with torch if not
    given (the library itself never allocates)."""
    import torch
    M, K = a.shape
    N, K2 = b_cols.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=a.device)
    elif tuple(out.shape) != (M, N):
        raise ValueError(f"out must be ({M}, {N})")
    hgemm(a, b_cols, out, M, N, K, stream)
    return out


# ------------------------------------------- the feed-forward block's operators

_F16, _F32, _I8, _U8 = "torch.float16", "torch.float32", "torch.int8", "torch.uint8"
_dtypes: dict = {}  # torch's dtype objects and their names


def _dev(x, dtype: str, name: str):
    """Address of a CUDA tensor of `dtype`; None and raw addresses pass."""
    if x is None or type(x) is int:
        return x
    if _dtypes.get(x.dtype) is not dtype:
        if str(x.dtype) != dtype:
            raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
        _dtypes[x.dtype] = dtype
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return x.data_ptr()


def hgemm_linear(X, ldx: int, W, ldw: int, bias, act: int, R, ldr: int, Y, ldy: int, M: int, N: int, K: int,
                 codes=None, ldq: int = 0, scales=None, lds: int = 0, stream=None) -> None:
    """Y = f(X·Wᵀ + bias) + R, f an HGEMM_ACT_*; with codes and scales the
    pre-activations are kept in 8 bits too (see hgemm.h)."""
    _raise_on((_lib or load()).hgemm_linear(
        _dev(X, _F16, "X"), ldx, _dev(W, _F16, "W"), ldw, _dev(bias, _F16, "bias"), act, _dev(R, _F16, "R"), ldr,
        _dev(Y, _F16, "Y"), ldy, _dev(codes, _I8, "codes"), ldq, _dev(scales, _F32, "scales"), lds, M, N, K,
        _stream(stream)), "hgemm_linear")


def hgemm_linear_dgrad(dY, lddy: int, W, ldw: int, codes, ldq: int, scales, lds: int, act: int, dU, lddu: int,
                       H, ldh: int, M: int, N: int, K: int, stream=None) -> None:
    """dU = (dY·W) ⊙ f'(Û) and H = f(Û), Û the 8-bit pre-activations (see hgemm.h)."""
    _raise_on((_lib or load()).hgemm_linear_dgrad(
        _dev(dY, _F16, "dY"), lddy, _dev(W, _F16, "W"), ldw, _dev(codes, _I8, "codes"), ldq,
        _dev(scales, _F32, "scales"), lds, act, _dev(dU, _F16, "dU"), lddu, _dev(H, _F16, "H"), ldh, M, N, K,
        _stream(stream)), "hgemm_linear_dgrad")


def hgemm_linear_wgrad(dY, lddy: int, X, ldx: int, dW, lddw: int, dbias, accumulate: bool, M: int, N: int, K: int,
                       stream=None) -> None:
    """dW = dYᵀ·X and dbias = Σ_rows dY, or added to both (see hgemm.h)."""
    _raise_on((_lib or load()).hgemm_linear_wgrad(
        _dev(dY, _F16, "dY"), lddy, _dev(X, _F16, "X"), ldx, _dev(dW, _F16, "dW"), lddw, _dev(dbias, _F32, "dbias"),
        1 if accumulate else 0, M, N, K, _stream(stream)), "hgemm_linear_wgrad")


def hgemm_layernorm_forward(X, ldx: int, gamma, beta, eps: float, Y, ldy: int, mean, rstd, M: int, D: int,
                            stream=None) -> None:
    """Y = (X − mean)·rstd·gamma + beta over rows of D values (see hgemm.h)."""
    _raise_on((_lib or load()).hgemm_layernorm_forward(
        _dev(X, _F16, "X"), ldx, _dev(gamma, _F16, "gamma"), _dev(beta, _F16, "beta"), eps, _dev(Y, _F16, "Y"), ldy,
        _dev(mean, _F32, "mean"), _dev(rstd, _F32, "rstd"), M, D, _stream(stream)), "hgemm_layernorm_forward")


def hgemm_layernorm_backward_workspace_size(M: int, D: int) -> int:
    """Bytes of device workspace hgemm_layernorm_backward needs."""
    return int(load().hgemm_layernorm_backward_workspace_size(M, D))


def hgemm_layernorm_backward(dY, lddy: int, X, ldx: int, gamma, mean, rstd, R, ldr: int, dX, lddx: int, dgamma,
                             dbeta, workspace, M: int, D: int, workspace_bytes: int | None = None,
                             stream=None) -> None:
    """dX, dgamma and dbeta of a layer norm, R added to dX (see hgemm.h); the
    workspace's size defaults to the tensor's bytes."""
    if workspace is not None and type(workspace) is not int and not getattr(workspace, "is_cuda", False):
        raise ValueError("workspace must be a CUDA tensor")
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    _raise_on((_lib or load()).hgemm_layernorm_backward(
        _dev(dY, _F16, "dY"), lddy, _dev(X, _F16, "X"), ldx, _dev(gamma, _F16, "gamma"), _dev(mean, _F32, "mean"),
        _dev(rstd, _F32, "rstd"), _dev(R, _F16, "R"), ldr, _dev(dX, _F16, "dX"), lddx, _dev(dgamma, _F32, "dgamma"),
        _dev(dbeta, _F32, "dbeta"), _ptr(workspace), workspace_bytes, M, D, _stream(stream)),
        "hgemm_layernorm_backward")


def hgemm_ckpt8_save(X, ldx: int, codes, ldq: int, scales, lds: int, M: int, N: int, stream=None) -> None:
    """X into its 8-bit form (see hgemm.h)."""
    _raise_on((_lib or load()).hgemm_ckpt8_save(
        _dev(X, _F16, "X"), ldx, _dev(codes, _I8, "codes"), ldq, _dev(scales, _F32, "scales"), lds, M, N,
        _stream(stream)), "hgemm_ckpt8_save")


def hgemm_ckpt8_load(codes, ldq: int, scales, lds: int, act: int, Y, ldy: int, M: int, N: int, stream=None) -> None:
    """Y = f(Û) from the 8-bit form, f an HGEMM_ACT_* (see hgemm.h)."""
    _raise_on((_lib or load()).hgemm_ckpt8_load(
        _dev(codes, _I8, "codes"), ldq, _dev(scales, _F32, "scales"), lds, act, _dev(Y, _F16, "Y"), ldy, M, N,
        _stream(stream)), "hgemm_ckpt8_load")


def _workspace(workspace, workspace_bytes):
    if workspace is not None and type(workspace) is not int and not getattr(workspace, "is_cuda", False):
        raise ValueError("workspace must be a CUDA tensor")
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    return _ptr(workspace), workspace_bytes


def hgemm_residual_norm_forward(X, ldx, alpha: float, Y, ldy, gate, post: int, post_gamma, post_beta, pre: int,
                                pre_gamma, pre_beta, eps: float, Z, ldz, H, ldh, stats, M: int, D: int,
                                stream=None) -> None:
    """Z = alpha·X + gate ⊙ N_post(Y) and H = N_pre(Z); the norms are HGEMM_NORM_* (see hgemm.h)."""
    _raise_on((_lib or load()).hgemm_residual_norm_forward(
        _dev(X, _F16, "X"), ldx, alpha, _dev(Y, _F16, "Y"), ldy, _dev(gate, _F16, "gate"), post,
        _dev(post_gamma, _F16, "post_gamma"), _dev(post_beta, _F16, "post_beta"), pre,
        _dev(pre_gamma, _F16, "pre_gamma"), _dev(pre_beta, _F16, "pre_beta"), eps, _dev(Z, _F16, "Z"), ldz,
        _dev(H, _F16, "H"), ldh, _dev(stats, _F32, "stats"), M, D, _stream(stream)), "hgemm_residual_norm_forward")


def hgemm_residual_norm_backward_workspace_size(M: int, D: int) -> int:
    """Bytes of device workspace hgemm_residual_norm_backward needs."""
    return int(load().hgemm_residual_norm_backward_workspace_size(M, D))


def hgemm_residual_norm_backward(dZ, lddz, dH, lddh, Z, ldz, Y, ldy, alpha: float, gate, post: int, post_gamma,
                                 post_beta, pre: int, pre_gamma, stats, dX, lddx, dY, lddy, dgate, dpost_gamma,
                                 dpost_beta, dpre_gamma, dpre_beta, workspace, M: int, D: int,
                                 workspace_bytes: int | None = None, stream=None) -> None:
    """dX, dY and the vectors' gradients of hgemm_residual_norm_forward (see
    hgemm.h); the workspace's size defaults to the tensor's bytes."""
    ws, nbytes = _workspace(workspace, workspace_bytes)
    _raise_on((_lib or load()).hgemm_residual_norm_backward(
        _dev(dZ, _F16, "dZ"), lddz, _dev(dH, _F16, "dH"), lddh, _dev(Z, _F16, "Z"), ldz, _dev(Y, _F16, "Y"), ldy,
        alpha, _dev(gate, _F16, "gate"), post, _dev(post_gamma, _F16, "post_gamma"),
        _dev(post_beta, _F16, "post_beta"), pre, _dev(pre_gamma, _F16, "pre_gamma"), _dev(stats, _F32, "stats"),
        _dev(dX, _F16, "dX"), lddx, _dev(dY, _F16, "dY"), lddy, _dev(dgate, _F32, "dgate"),
        _dev(dpost_gamma, _F32, "dpost_gamma"), _dev(dpost_beta, _F32, "dpost_beta"),
        _dev(dpre_gamma, _F32, "dpre_gamma"), _dev(dpre_beta, _F32, "dpre_beta"), ws, nbytes, M, D, _stream(stream)),
        "hgemm_residual_norm_backward")


# ---------------------------------------------------------------- the optimizer

class _AdamwTensor(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("master", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("n", ctypes.c_int64), ("weight_decay", ctypes.c_float),
                ("grad_type", ctypes.c_int32)]


class AdamwTensors:
    """The table of tensors that hgemm_adamw steps: their addresses, and the
    tensors themselves so that they stay alive. device: the CUDA device's number
    that gradients must be on; None: the first gradient's."""

    def __init__(self, table, keep, grads=(), device=None):
        self.table, self.keep, self.grads, self.device = table, keep, grads, device

    def set_gradients(self, grads) -> None:
        """Other gradients (float16 or float32) in place of the table's, in its
        order, checked as hgemm_adamw_tensors checks them: what a step without
        kept gradients changes. A refused call changes nothing."""
        import torch
        f16, f32 = torch.float16, torch.float32
        grads, table = list(grads), type(self.table).from_buffer_copy(self.table)
        if len(grads) != len(table):
            raise ValueError(f"{len(table)} gradients are needed, got {len(grads)}")
        device = self.device
        for i, (row, g) in enumerate(zip(table, grads)):
            dtype = g.dtype
            if dtype is not f16 and dtype is not f32:
                raise TypeError(f"tensor {i}: grad must be float16 or float32, got {dtype}")
            at = g.get_device()  # (−1 of a tensor on the host)
            if device is None:
                device = at
            if at != device or at < 0:
                raise ValueError(f"tensor {i}: grad must be on {'cuda' if device < 0 else f'cuda:{device}'}, got {g.device}")
            if g.numel() != row.n or not g.is_contiguous():
                raise ValueError(f"tensor {i}: grad must be {row.n} values, contiguous, got {tuple(g.shape)}")
            row.grad, row.grad_type = g.data_ptr(), HGEMM_TYPE_F16 if dtype is f16 else HGEMM_TYPE_F32
        _raise_on((_lib or load()).hgemm_adamw_check(table, len(table)), "hgemm_adamw_check")
        self.table, self.grads = table, grads


_ADAMW_FIELDS = {"weight", "master", "grad", "m", "v", "m_scales", "v_scales", "weight_decay"}


def hgemm_adamw_tensors(tensors) -> AdamwTensors:
    """The table for hgemm_adamw from dicts of CUDA tensors: ``grad`` (float16
    or float32), ``weight`` (float16) and ``master`` (float32) or either, the
    states ``m`` and ``v`` (float32; or int8 and uint8 with ``m_scales`` and
    ``v_scales``, float32, one per 64 values), and ``weight_decay`` (0 where not
    given). Made once for a program's tensors (set_gradients takes a later step's
    gradients); all contiguous, of equal size, on
    one device, and none may share memory with another's outputs."""
    import torch
    f16, f32, i8, u8 = torch.float16, torch.float32, torch.int8, torch.uint8
    tensors = list(tensors)
    rows, keep, device = [], [], None
    for i, t in enumerate(tensors):
        get = t.get
        grad = get("grad")
        if not t.keys() <= _ADAMW_FIELDS:
            raise TypeError(f"tensor {i}: unknown {sorted(set(t) - _ADAMW_FIELDS)}")
        for name in ("grad", "m", "v"):
            if get(name) is None:
                raise ValueError(f"tensor {i}: {name} is missing")
        eight = get("m_scales") is not None or get("v_scales") is not None
        n, groups = grad.numel(), 0
        if eight:
            groups = -(-n // HGEMM_CKPT8_GROUP)
        half_grad = grad.dtype is f16
        row = []
        for name, dtype, size in (("weight", f16, n), ("master", f32, n), ("grad", f16 if half_grad else f32, n),
                                  ("m", i8 if eight else f32, n), ("v", u8 if eight else f32, n),
                                  ("m_scales", f32, groups), ("v_scales", f32, groups)):
            x = get(name)
            if x is None:
                row.append(None)
                continue
            if x.dtype is not dtype:
                raise TypeError(f"tensor {i}: {name} must be {dtype}, got {x.dtype}")
            at = x.get_device()
            if at != device:
                if at < 0:
                    raise ValueError(f"tensor {i}: {name} must be a CUDA tensor")
                if device is not None:
                    raise ValueError(f"tensor {i}: {name} must be on cuda:{device}, got cuda:{at}")
                device = at
            if x.numel() != size or not x.is_contiguous():
                raise ValueError(f"tensor {i}: {name} must be {size} values, contiguous, got {tuple(x.shape)}")
            row.append(x.data_ptr())
            if name != "grad":
                keep.append(x)
        rows.append((*row, n, get("weight_decay", 0.0), HGEMM_TYPE_F16 if half_grad else HGEMM_TYPE_F32))
    plan = AdamwTensors((_AdamwTensor * len(rows))(*rows), keep, [t["grad"] for t in tensors], device)
    hgemm_adamw_check(plan)
    return plan


def hgemm_adamw_check(tensors: AdamwTensors) -> None:
    """Raises where hgemm_adamw would refuse a tensor, and where one's arrays
    overlap another's outputs (hgemm_adamw_tensors has called it)."""
    _raise_on((_lib or load()).hgemm_adamw_check(tensors.table, len(tensors.table)), "hgemm_adamw_check")


def hgemm_adamw_dynamic(lr: float, grad_scale: float, step: int, skip: bool = False):
    """The 16 bytes of an hgemm_adamw_dynamic as a host tensor of bytes, to be
    copied to the device tensor that a captured step reads."""
    import struct
    import torch
    return torch.frombuffer(bytearray(struct.pack("=ffii", lr, grad_scale, step, 1 if skip else 0)), dtype=torch.uint8)


def hgemm_adamw(tensors: AdamwTensors, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                step: int = 1, grad_scale: float = 1.0, dynamic=None, stream=None) -> None:
    """One AdamW step over the tensors of hgemm_adamw_tensors (see hgemm.h), 8-bit
    states rounded to nearest: carried over many steps they stop following their
    gradients, where hgemm_adamw_rounded is for. dynamic: 16 device bytes
    (hgemm_adamw_dynamic's) that are read when the step runs, or None."""
    hgemm_adamw_rounded(tensors, lr, beta1, beta2, eps, step, grad_scale, HGEMM_ROUND_NEAREST, dynamic, stream)


def hgemm_adamw_rounded(tensors: AdamwTensors, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                        step: int = 1, grad_scale: float = 1.0, rounding: int = HGEMM_ROUND_RANDOM, dynamic=None,
                        stream=None) -> None:
    """hgemm_adamw with a choice of how 8-bit states are rounded, HGEMM_ROUND_*:
    at random is what training takes (see hgemm.h)."""
    if dynamic is not None and type(dynamic) is not int:
        if not getattr(dynamic, "is_cuda", False):
            raise ValueError("dynamic must be a CUDA tensor")
        if dynamic.numel() * dynamic.element_size() < 16 or not dynamic.is_contiguous():
            raise ValueError("dynamic must have 16 bytes, contiguous")
    if tensors.device is not None or stream is None:
        current = (_torch or _import_torch()).cuda.current_device()
        if tensors.device is not None and tensors.device != current:
            raise ValueError(f"the tensors are on cuda:{tensors.device}, the current device is cuda:{current}")
        if stream is None:
            stream = int(_raw_current_stream(current))
    _raise_on((_lib or load()).hgemm_adamw_rounded(tensors.table, len(tensors.table), lr, beta1, beta2, eps, step,
                                                   grad_scale, rounding, _ptr(dynamic), _stream(stream)),
              "hgemm_adamw_rounded")


def hgemm_adamw_load(m, m_scales, v, v_scales, m_out, v_out, n: int, stream=None) -> None:
    """8-bit states read back as float32 (see hgemm.h)."""
    _raise_on((_lib or load()).hgemm_adamw_load(
        _dev(m, _I8, "m"), _dev(m_scales, _F32, "m_scales"), _dev(v, _U8, "v"),
        _dev(v_scales, _F32, "v_scales"), _dev(m_out, _F32, "m_out"), _dev(v_out, _F32, "v_out"), n, _stream(stream)),
        "hgemm_adamw_load")


# ------------------------------------------------------------ mixture of experts

def hgemm_experts_workspace_size(M: int, D: int, F: int, E: int, k: int) -> int:
    """Bytes of device workspace hgemm_experts needs."""
    return int(load().hgemm_experts_workspace_size(M, D, F, E, k))


def hgemm_experts(X, ldx, Wr, ldwr, W1, ldw1, b1, W2, ldw2, b2, act: int, gated: bool, k: int, normalize: bool, R, ldr,
                  Y, ldy, chosen, share, workspace, M: int, D: int, F: int, E: int,
                  workspace_bytes: int | None = None, stream=None) -> None:
    """Y = Σ s·(W2·f(W1·x + b1) + b2) + R over the k experts of E that the
    router Wr chooses for each of M tokens (see hgemm.h); the workspace's size
    defaults to the tensor's bytes."""
    ws, nbytes = _workspace(workspace, workspace_bytes)
    _raise_on((_lib or load()).hgemm_experts(
        _dev(X, _F16, "X"), ldx, _dev(Wr, _F16, "Wr"), ldwr, _dev(W1, _F16, "W1"), ldw1, _dev(b1, _F16, "b1"),
        _dev(W2, _F16, "W2"), ldw2, _dev(b2, _F16, "b2"), act, 1 if gated else 0, k, 1 if normalize else 0,
        _dev(R, _F16, "R"), ldr, _dev(Y, _F16, "Y"), ldy, _dev(chosen, "torch.int32", "chosen"),
        _dev(share, _F32, "share"), ws, nbytes, M, D, F, E, _stream(stream)), "hgemm_experts")
