"""ctypes binding of the C ABI in include/nvfp4_moe.h.

Argument marshalling only, with the C entry points' names; addresses are
device addresses as integers (0: NULL). The library must have been built
(``python -m moe_matmul_amd.build``); there is no fallback. Tensors are taken by
``moe_matmul_amd.moe``.
"""
from __future__ import annotations

import ctypes
import functools
import os

from ._binding import NVFP4_ERR_HIP, NVFP4_OK, Nvfp4Error, nvfp4_error_string

MOE_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4_moe.so")

NVFP4_MOE_F32, NVFP4_MOE_F16, NVFP4_MOE_BF16 = 0, 1, 2
NVFP4_MOE_SOFTMAX, NVFP4_MOE_SIGMOID = 0, 1
NVFP4_MOE_MAX_EXPERTS = 512
NVFP4_MOE_MAX_TOPK = 16
NVFP4_MOE_MAX_GROUPS = 64
NVFP4_MOE_MAX_FEW_SLOTS = 4096
NVFP4_MOE_MAX_PRODUCTS = 4


class Nvfp4MoeError(Nvfp4Error):
    def __init__(self, code: int, what: str):
        self.code = code
        RuntimeError.__init__(self, f"{what} failed: {code} ({nvfp4_error_string(code)})"
                              + (f", hip error {nvfp4_moe_last_hip_error()}" if code == NVFP4_ERR_HIP else ""))


class nvfp4_moe_choice(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("topk", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("group_best", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class nvfp4_moe_product(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("k", ctypes.c_int32)] + [
        (name, ctypes.c_uint64) for name in ("a", "b", "c", "sfa", "sfb", "sizes", "abc", "sf")]


_int, _i64, _float, _ptr, _size = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
_choice, _products = ctypes.POINTER(nvfp4_moe_choice), ctypes.POINTER(nvfp4_moe_product)
_SIGNATURES = {
    "nvfp4_moe_route": (_int, [_ptr, _int, _i64, _int, _i64, _ptr, _choice, _ptr, _ptr, _ptr]),
    "nvfp4_moe_route_backward": (_int, [_ptr, _int, _i64, _int, _i64, _choice, _ptr, _ptr, _ptr, _i64, _ptr]),
    "nvfp4_moe_plan": (_int, [_ptr, _i64, _int, _int, _ptr, _ptr, _ptr, _ptr, _products, _int, _ptr, _size, _ptr]),
    "nvfp4_moe_plan_ex": (_int, [_ptr, _i64, _int, _int, _ptr, _ptr, _ptr, _ptr, _ptr, _products, _int, _ptr, _size, _ptr]),
    "nvfp4_moe_plan_workspace_bytes": (_size, [_i64, _int, _int]),
    "nvfp4_moe_sf_bytes": (_size, [_i64, _int, _int]),
    "nvfp4_moe_quantize": (_int, [_ptr, _int, _int, _i64, _int, _i64, _i64, _float, _ptr, _ptr, _ptr]),
    "nvfp4_moe_dispatch": (_int, [_ptr, _int, _i64, _int, _int, _i64, _float, _ptr, _ptr, _ptr, _ptr, _ptr, _int,
                                  _ptr, _ptr, _ptr, _size, _ptr]),
    "nvfp4_moe_dispatch_workspace_bytes": (_size, [_i64, _int, _int]),
    "nvfp4_moe_swiglu": (_int, [_ptr, _int, _i64, _int, _i64, _ptr, _float, _ptr, _ptr, _int, _ptr, _ptr, _ptr]),
    "nvfp4_moe_dequantize": (_int, [_ptr, _ptr, _int, _i64, _int, _ptr, _ptr, _int, _ptr, _int, _i64, _ptr]),
    "nvfp4_moe_combine": (_int, [_ptr, _int, _i64, _i64, _i64, _int, _int, _ptr, _ptr, _ptr, _ptr, _int, _ptr, _ptr, _int,
                                 _i64, _ptr]),
    "nvfp4_moe_combine_backward": (_int, [_ptr, _int, _i64, _ptr, _int, _i64, _i64, _i64, _int, _int, _ptr, _ptr, _ptr,
                                          _ptr, _int, _ptr, _ptr, _ptr]),
    "nvfp4_moe_few_tokens": (_int, [_ptr, _int, _i64, _int, _ptr, _i64, _int, _int, _int, _int, _ptr, _ptr, _ptr,
                                    _int, _ptr, _int, _ptr]),
    "nvfp4_moe_last_hip_error": (_int, []),
}

_lib = None


def load_moe_library() -> ctypes.CDLL:
    """Load the built library (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(MOE_LIB_PATH):
            raise ImportError(f"{MOE_LIB_PATH} is not built: run `python -m moe_matmul_amd.build` "
                              "(these operators have no non-HIP implementation)")
        lib = ctypes.CDLL(MOE_LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def _checked(name):
    def call(*args) -> None:
        rc = getattr(_lib or load_moe_library(), name)(*args)
        if rc != NVFP4_OK:
            raise Nvfp4MoeError(rc, name)
    call.__name__ = name
    call.__doc__ = f"{name} of include/nvfp4_moe.h, argument for argument; raises Nvfp4MoeError unless it returns NVFP4_OK."
    return call


nvfp4_moe_route = _checked("nvfp4_moe_route")
nvfp4_moe_route_backward = _checked("nvfp4_moe_route_backward")
nvfp4_moe_plan = _checked("nvfp4_moe_plan")
nvfp4_moe_plan_ex = _checked("nvfp4_moe_plan_ex")
nvfp4_moe_quantize = _checked("nvfp4_moe_quantize")
nvfp4_moe_dispatch = _checked("nvfp4_moe_dispatch")
nvfp4_moe_swiglu = _checked("nvfp4_moe_swiglu")
nvfp4_moe_dequantize = _checked("nvfp4_moe_dequantize")
nvfp4_moe_combine = _checked("nvfp4_moe_combine")
nvfp4_moe_combine_backward = _checked("nvfp4_moe_combine_backward")
nvfp4_moe_few_tokens = _checked("nvfp4_moe_few_tokens")


@functools.lru_cache(maxsize=4096)
def nvfp4_moe_plan_workspace_bytes(tokens: int, topk: int, experts: int) -> int:
    return load_moe_library().nvfp4_moe_plan_workspace_bytes(tokens, topk, experts)


@functools.lru_cache(maxsize=4096)
def nvfp4_moe_dispatch_workspace_bytes(tokens: int, topk: int, k: int) -> int:
    return load_moe_library().nvfp4_moe_dispatch_workspace_bytes(tokens, topk, k)


@functools.lru_cache(maxsize=4096)
def nvfp4_moe_sf_bytes(rows: int, experts: int, k: int) -> int:
    return load_moe_library().nvfp4_moe_sf_bytes(rows, experts, k)


def nvfp4_moe_last_hip_error() -> int:
    return load_moe_library().nvfp4_moe_last_hip_error()
