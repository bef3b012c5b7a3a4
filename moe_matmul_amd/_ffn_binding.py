"""ctypes binding of the C ABI in include/nvfp4_ffn.h.

Argument marshalling only, with the C entry points' names; addresses are
device addresses as integers (0: NULL). The library must have been built
(``python -m moe_matmul_amd.build``); there is no fallback. Tensors are taken by
``moe_matmul_amd.ffn``.
"""
from __future__ import annotations

import ctypes
import functools
import os

from ._binding import NVFP4_ERR_HIP, NVFP4_OK, Nvfp4Error, nvfp4_error_string

FFN_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4_ffn.so")

NVFP4_FFN_NONE, NVFP4_FFN_RELU, NVFP4_FFN_SILU, NVFP4_FFN_GELU = 0, 1, 2, 3
NVFP4_FFN_FORWARD, NVFP4_FFN_FORWARD_CODES, NVFP4_FFN_DX, NVFP4_FFN_DW = 0, 1, 2, 3


class Nvfp4FfnError(Nvfp4Error):
    def __init__(self, code: int, what: str):
        self.code = code
        RuntimeError.__init__(self, f"{what} failed: {code} ({nvfp4_error_string(code)})"
                              + (f", hip error {nvfp4_ffn_last_hip_error()}" if code == NVFP4_ERR_HIP else ""))


class nvfp4_ffn_plan(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int32), ("topk", ctypes.c_int32), ("offsets", ctypes.c_void_p),
                ("row_slots", ctypes.c_void_p)]


_int, _i64, _float, _ptr, _size = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
_plan = ctypes.POINTER(nvfp4_ffn_plan)
_SIGNATURES = {
    "nvfp4_ffn_rmsnorm": (_int, [_ptr, _int, _i64, _int, _i64, _ptr, _i64, _ptr, _int, _float, _ptr, _ptr, _ptr, _ptr,
                                 _ptr, _ptr]),
    "nvfp4_ffn_rmsnorm_backward": (_int, [_ptr, _i64, _ptr, _i64, _int, _i64, _int, _ptr, _int, _ptr, _ptr, _i64, _ptr,
                                          _ptr, _ptr, _size, _ptr]),
    "nvfp4_ffn_rmsnorm_workspace_bytes": (_size, [_i64, _int]),
    "nvfp4_ffn_quantize8": (_int, [_ptr, _int, _i64, _int, _i64, _ptr, _ptr, _ptr]),
    "nvfp4_ffn_dequantize8": (_int, [_ptr, _ptr, _i64, _int, _ptr, _int, _i64, _ptr]),
    "nvfp4_ffn_gather": (_int, [_ptr, _i64, _ptr, _ptr, _int, _i64, _int, _plan, _ptr, _ptr]),
    "nvfp4_ffn_linear": (_int, [_ptr, _i64, _ptr, _ptr, _int, _int, _ptr, _i64, _ptr, _ptr, _int, _i64, _int, _int, _plan,
                                _int, _ptr, _size, _ptr]),
    "nvfp4_ffn_gated": (_int, [_ptr, _i64, _ptr, _int, _ptr, _ptr, _ptr, _ptr, _int, _i64, _int, _int, _plan, _int, _ptr,
                               _size, _ptr]),
    "nvfp4_ffn_product_workspace_bytes": (_size, [_i64, _int, _int, _int]),
    "nvfp4_ffn_product_parts": (_int, [_int, _i64, _int, _int, _int, ctypes.POINTER(ctypes.c_int32)]),
    "nvfp4_ffn_linear_dz": (_int, [_ptr, _i64, _ptr, _int, _ptr, _ptr, _int, _int, _i64, _int, _plan, _ptr, _size, _ptr]),
    "nvfp4_ffn_dz_workspace_bytes": (_size, [_i64, _int, _int]),
    "nvfp4_ffn_gated_dz": (_int, [_ptr, _i64, _ptr, _ptr, _ptr, _int, _ptr, _int, _i64, _int, _plan, _ptr]),
    "nvfp4_ffn_gated_again": (_int, [_ptr, _i64, _ptr, _i64, _ptr, _int, _ptr, _int, _i64, _int, _int, _plan, _ptr, _size,
                                     _ptr]),
    "nvfp4_ffn_linear_dx": (_int, [_ptr, _i64, _ptr, _ptr, _int, _i64, _int, _int, _plan, _int, _ptr, _size, _ptr]),
    "nvfp4_ffn_linear_dx_ex": (_int, [_ptr, _i64, _ptr, _ptr, _int, _int, _i64, _int, _int, _plan, _int, _ptr, _size, _ptr]),
    "nvfp4_ffn_linear_dw": (_int, [_ptr, _i64, _ptr, _i64, _ptr, _int, _int, _i64, _int, _int, _plan, _ptr, _size, _ptr]),
    "nvfp4_ffn_dw_workspace_bytes": (_size, [_i64, _int, _int, _int]),
    "nvfp4_ffn_last_hip_error": (_int, []),
}

_lib = None


def load_ffn_library() -> ctypes.CDLL:
    """Load the built library (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(FFN_LIB_PATH):
            raise ImportError(f"{FFN_LIB_PATH} is not built: run `python -m moe_matmul_amd.build` "
                              "(these operators have no non-HIP implementation)")
        lib = ctypes.CDLL(FFN_LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def _checked(name):
    def call(*args) -> None:
        rc = getattr(_lib or load_ffn_library(), name)(*args)
        if rc != NVFP4_OK:
            raise Nvfp4FfnError(rc, name)
    call.__name__ = name
    call.__doc__ = f"{name} of include/nvfp4_ffn.h, argument for argument; raises Nvfp4FfnError unless it returns NVFP4_OK."
    return call


nvfp4_ffn_rmsnorm = _checked("nvfp4_ffn_rmsnorm")
nvfp4_ffn_rmsnorm_backward = _checked("nvfp4_ffn_rmsnorm_backward")
nvfp4_ffn_quantize8 = _checked("nvfp4_ffn_quantize8")
nvfp4_ffn_dequantize8 = _checked("nvfp4_ffn_dequantize8")
nvfp4_ffn_gather = _checked("nvfp4_ffn_gather")
nvfp4_ffn_linear = _checked("nvfp4_ffn_linear")
nvfp4_ffn_gated = _checked("nvfp4_ffn_gated")
nvfp4_ffn_linear_dz = _checked("nvfp4_ffn_linear_dz")
nvfp4_ffn_gated_dz = _checked("nvfp4_ffn_gated_dz")
nvfp4_ffn_gated_again = _checked("nvfp4_ffn_gated_again")
nvfp4_ffn_linear_dx = _checked("nvfp4_ffn_linear_dx")
nvfp4_ffn_linear_dx_ex = _checked("nvfp4_ffn_linear_dx_ex")
nvfp4_ffn_linear_dw = _checked("nvfp4_ffn_linear_dw")


# Buffer sizes, kept by the index of the device whose compute units go into them: it has to be the current one.
@functools.lru_cache(maxsize=4096)
def nvfp4_ffn_rmsnorm_workspace_bytes(rows: int, n: int, device: int = 0) -> int:
    return load_ffn_library().nvfp4_ffn_rmsnorm_workspace_bytes(rows, n)


@functools.lru_cache(maxsize=4096)
def nvfp4_ffn_product_workspace_bytes(rows: int, n: int, k: int, experts: int, device: int = 0) -> int:
    return load_ffn_library().nvfp4_ffn_product_workspace_bytes(rows, n, k, experts)


@functools.lru_cache(maxsize=4096)
def nvfp4_ffn_dz_workspace_bytes(rows: int, n: int, experts: int, device: int = 0) -> int:
    return load_ffn_library().nvfp4_ffn_dz_workspace_bytes(rows, n, experts)


@functools.lru_cache(maxsize=4096)
def nvfp4_ffn_dw_workspace_bytes(rows: int, n: int, k: int, experts: int, device: int = 0) -> int:
    return load_ffn_library().nvfp4_ffn_dw_workspace_bytes(rows, n, k, experts)


def nvfp4_ffn_product_parts(kind: int, rows: int, n: int, k: int, experts: int) -> list:
    """[(rows, tile rows, tile columns, parts of k)] of a product's launches; a tile of (0, 0): the kernel of few rows."""
    out = (ctypes.c_int32 * 8)()
    count = load_ffn_library().nvfp4_ffn_product_parts(kind, rows, n, k, experts, out)
    return [tuple(out[4 * i:4 * i + 4]) for i in range(count)]


def nvfp4_ffn_last_hip_error() -> int:
    return load_ffn_library().nvfp4_ffn_last_hip_error()
