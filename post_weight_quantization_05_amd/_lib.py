"""ctypes declarations of libqz (include/qz.h).  Loading fails loudly when the built
library is missing: there is no fallback implementation."""
from __future__ import annotations

import ctypes as C
import os
import warnings

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqz.so")

QZ_OK, QZ_EINVAL, QZ_ENOTPD, QZ_ENONFINITE, QZ_EHIP, QZ_ESOLVER, QZ_EWORKSPACE = 0, -1, -2, -3, -4, -5, -6
QZ_BF16, QZ_F32 = 0, 1
QZ_GRID_CALLER = 0x1
QZ_H_ACCUMULATE = 0x1
QZ_H_NO_FINALIZE = 0x2
QZ_ADMM_WARM_START = 0x1
QZ_ADMM_REFRESH_UNCLAMPED = 0x2
QZ_ADMM_REFRESH_FROM_Z = 0x4
QZ_ADMM_DUAL_NO_RESCALE = 0x8
QZ_ORDER_ACT = 1
QZ_ORDER_MIN_PIVOT = 2
QZ_MX4_FLOOR, QZ_MX4_LEAST = 0, 1
QZ_MOE_RENORM = 0x1
QZ_ROUTE_SIGMOID, QZ_ROUTE_RENORM = 0x1, 0x2
QZ_I8_MAX_COLS = 65536

STATUS_NAMES = {0: "QZ_OK", -1: "QZ_EINVAL", -2: "QZ_ENOTPD", -3: "QZ_ENONFINITE", -4: "QZ_EHIP",
                -5: "QZ_ESOLVER", -6: "QZ_EWORKSPACE"}

# every entry point declared in include/qz.h
EXPORTS = ("qz_hessian_workspace", "qz_build_hessian", "qz_rtn_workspace", "qz_rtn",
           "qz_rtn_noalloc",
           "qz_gptq_workspace", "qz_gptq",
           "qz_gptq_noclip", "qz_order_workspace", "qz_order", "qz_error_bound_workspace",
           "qz_error_bound",
           "qz_admmq_prepare_workspace", "qz_admmq_prepare", "qz_admmq_workspace", "qz_admmq", "qz_objective_workspace",
           "qz_objective", "qz_objective_i32", "qz_local_search_workspace", "qz_local_search",
           "qz_packed_words",
           "qz_pack",
           "qz_unpack",
           "qz_mx4_blocks", "qz_mx4_quantize", "qz_mx4_unpack", "qz_mx4_linear_workspace",
           "qz_mx4_linear", "qz_mx4_matmul_workspace", "qz_mx4_matmul", "qz_mx4_moe_workspace",
           "qz_mx4_moe",
           "qz_i8_pitch", "qz_i8_quantize", "qz_i8_pack", "qz_i8_unpack", "qz_i8_matmul_workspace",
           "qz_i8_matmul", "qz_i8_linear_workspace", "qz_i8_linear", "qz_route",
           "qz_i8_moe_workspace", "qz_i8_moe",
           "qz_timing_enable", "qz_timing_read", "qz_timing_kind_name",
           "qz_last_error", "qz_abi_version")


class QzGrid(C.Structure):
    _fields_ = [("struct_size", C.c_uint32), ("bits", C.c_int32), ("group_size", C.c_int32),
                ("flags", C.c_uint32)]


class QzAdmm(C.Structure):
    _fields_ = [("struct_size", C.c_uint32), ("iters", C.c_int32), ("rho0", C.c_float),
                ("gamma", C.c_float), ("refresh_every", C.c_int32), ("flags", C.c_uint32),
                ("t0", C.c_int32)]


class QzMoe(C.Structure):
    _fields_ = [("struct_size", C.c_uint32), ("n_experts", C.c_int32), ("top_k", C.c_int32),
                ("flags", C.c_uint32)]


class QzRouter(C.Structure):
    _fields_ = [("struct_size", C.c_uint32), ("n_experts", C.c_int32), ("top_k", C.c_int32),
                ("n_groups", C.c_int32), ("top_groups", C.c_int32), ("group_best", C.c_int32),
                ("flags", C.c_uint32), ("scale", C.c_float)]


P = C.c_void_p
I64 = C.c_int64
I32 = C.c_int32
U32 = C.c_uint32
SZ = C.c_size_t
F = C.c_float

_SIGS = {
    "qz_hessian_workspace": (SZ, [I64, I64, I32]),
    "qz_build_hessian": (C.c_int, [P, I32, I64, I64, F, U32, P, P, P, P, P, P, SZ, P]),
    "qz_rtn_workspace": (SZ, [I64, I64]),
    "qz_rtn": (C.c_int, [P, I32, I64, I64, C.POINTER(QzGrid), P, P, P, P, SZ, P]),
    "qz_rtn_noalloc": (C.c_int, [P, I32, I64, I64, C.POINTER(QzGrid), P, P, P, P]),
    "qz_gptq_workspace": (SZ, [I64, I64, I32]),
    "qz_gptq": (C.c_int, [P, P, I32, I64, I64, C.POINTER(QzGrid), I32, P, P, P, P, P, SZ, P]),
    "qz_gptq_noclip": (C.c_int, [P, P, I32, I64, I64, C.POINTER(QzGrid), I32, P, P, P, P, P, SZ,
                                 P]),
    "qz_order_workspace": (SZ, [I64, I32]),
    "qz_order": (C.c_int, [P, I64, I32, P, P, P, SZ, P]),
    "qz_error_bound_workspace": (SZ, [I64, I64]),
    "qz_error_bound": (C.c_int, [P, I64, P, P, I64, I32, P, P, P, SZ, P]),
    "qz_admmq_prepare_workspace": (SZ, [I64]),
    "qz_admmq_prepare": (C.c_int, [P, I64, P, P, P, P, SZ, P]),
    "qz_admmq_workspace": (SZ, [I64, I64, I32, I32]),
    "qz_admmq": (C.c_int, [P, P, P, P, I32, I64, I64, C.POINTER(QzGrid), C.POINTER(QzAdmm), P, P, P,
                           P, P, P, SZ, P]),
    "qz_objective_workspace": (SZ, [I64, I64]),
    "qz_objective": (C.c_int, [P, P, I32, P, P, P, I64, I64, I32, P, P, P, SZ, P]),
    "qz_objective_i32": (C.c_int, [P, P, I32, P, P, P, I64, I64, I32, P, P, P, SZ, P]),
    "qz_local_search_workspace": (SZ, [I64, I64, I32]),
    "qz_local_search": (C.c_int, [P, P, I32, I64, I64, C.POINTER(QzGrid), P, P, P, I32, P, P, P,
                                  SZ, P]),
    "qz_packed_words": (I64, [I64, I32]),
    "qz_pack": (C.c_int, [P, I64, I64, I32, P, P]),
    "qz_unpack": (C.c_int, [P, I64, I64, I32, P, P]),
    "qz_mx4_blocks": (I64, [I64]),
    "qz_mx4_quantize": (C.c_int, [P, I32, I64, I64, I64, I32, P, P, P, P, P]),
    "qz_mx4_unpack": (C.c_int, [P, P, I64, I64, P, P, P, P]),
    "qz_mx4_linear_workspace": (SZ, [P, I64, I64, I64, I64]),
    "qz_mx4_linear": (C.c_int, [P, I32, I64, I64, P, P, I64, I64, P, P, I32, I64, P, SZ, P]),
    "qz_mx4_matmul_workspace": (SZ, [I64, I64, I64]),
    "qz_mx4_matmul": (C.c_int, [P, P, I64, P, P, I64, I64, P, P, I32, I64, P, SZ, P]),
    "qz_mx4_moe_workspace": (SZ, [I64, I64, I64, C.POINTER(QzMoe)]),
    "qz_mx4_moe": (C.c_int, [P, I32, I64, I64, I64, I64, C.POINTER(QzMoe), P, I32, P, P, P, P, P, P,
                             P, P, SZ, P]),
    "qz_i8_pitch": (I64, [I64]),
    "qz_i8_quantize": (C.c_int, [P, I32, I64, I64, I64, P, P, P, P, P, P]),
    "qz_i8_pack": (C.c_int, [P, I64, I64, P, P]),
    "qz_i8_unpack": (C.c_int, [P, I64, I64, P, P]),
    "qz_i8_matmul_workspace": (SZ, [I64, I64, I64]),
    "qz_i8_matmul": (C.c_int, [P, P, P, I64, P, P, P, I64, I64, P, P, I32, I64, P, SZ, P]),
    "qz_i8_linear_workspace": (SZ, [I64, I64, I64]),
    "qz_i8_linear": (C.c_int, [P, I32, I64, I64, P, P, P, P, I64, I64, P, P, I32, I64, P, SZ, P]),
    "qz_route": (C.c_int, [P, I32, I64, I64, C.POINTER(QzRouter), P, P, P, P]),
    "qz_i8_moe_workspace": (SZ, [I64, I64, I64, I32, I32]),
    "qz_i8_moe": (C.c_int, [P, I32, I64, I64, I64, I64, I32, I32, P, P, P, P, P, P, P, P, P, P, SZ, P]),
    "qz_timing_enable": (C.c_int, [C.c_int]),
    "qz_timing_read": (C.c_int, [C.POINTER(C.c_int64), C.POINTER(C.c_double), C.c_int, C.c_int]),
    "qz_timing_kind_name": (C.c_char_p, [C.c_int]),
    "qz_last_error": (C.c_char_p, []),
    "qz_abi_version": (C.c_int, []),
}

_lib = None
binding = None      # the native calls (csrc/binding.cpp); None: every call through ctypes, to the same library
_BINDING_ORDER = ("qz_i8_quantize", "qz_i8_matmul_workspace", "qz_i8_matmul", "qz_i8_linear_workspace",
                  "qz_i8_linear", "qz_route", "qz_i8_moe_workspace", "qz_i8_moe")


def _native_calls(lib):
    """The binding module bound to `lib`; None where it is not built, or (with a warning) cannot be loaded here: one
    of another Python, PyTorch or ABI version must not take the library with it."""
    if not os.path.exists(os.path.join(_HERE, "_binding.so")):
        return None
    try:
        from . import _binding
        _binding.init(lib.qz_abi_version(), *(C.cast(getattr(lib, name), C.c_void_p).value for name in _BINDING_ORDER))
        return _binding
    except Exception as e:
        warnings.warn(f"_binding.so is not usable ({e}): calls go through ctypes; rebuild the package", RuntimeWarning,
                      stacklevel=3)
        return None


def load(path: str = LIB_PATH):
    """Load libqz.so and declare its signatures.  Raises if it is not built."""
    global _lib, binding
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libqz.so not found at {path}; build it with "
                          f"`python -m post_weight_quantization_05_amd.build`")
    # PyTorch ships its own HIP runtime and loads it by path.  Importing torch first
    # makes libqz's libamdhip64.so.7 dependency resolve (by soname) to that same
    # runtime, so device pointers and streams from torch are valid in libqz.  Loading
    # libqz first would bring up a second, separate HIP runtime in the process.
    import torch  # noqa: F401
    lib = C.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    binding = _native_calls(lib)
    return lib
