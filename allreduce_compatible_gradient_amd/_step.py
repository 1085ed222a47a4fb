"""libgq_step.so (``include/gq_step.h``): its signatures, loading and errors,
for ``fp8`` and ``optim``."""
from __future__ import annotations

import ctypes
import os

from . import GQError

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgq_step.so")


class CTensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_exps", ctypes.c_void_p), ("v_exps", ctypes.c_void_p),
                ("n", ctypes.c_int64)]


class CAdamWArgs(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("step", ctypes.c_int64), ("scale", ctypes.c_void_p),
                ("lr_device", ctypes.c_void_p), ("step_device", ctypes.c_void_p),
                ("seed", ctypes.c_uint64), ("random", ctypes.c_int32), ("bits", ctypes.c_int32)]


_i32, _i64, _u64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p
_f64 = ctypes.c_double
_args = ctypes.POINTER(CAdamWArgs)
# a list of tensors goes in as an array of 64-bit words, seven to a tensor
SIGNATURES = {
    "gqs_fp8_blocks": (_i64, [_i64]),
    "gqs_fp8_pitch": (_i64, [_i64]),
    "gqs_fp8_exp_pitch": (_i64, [_i64]),
    "gqs_fp8_rows": (_i32, [_vp, _i32, _i64, _i64, _i64, _i32, _u64, _vp, _vp, _vp]),
    "gqs_fp8_weight": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "gqs_fp8_restore": (_i32, [_vp, _vp, _i64, _i64, _i32, _i32, _vp, _vp]),
    "gqs_fp8_product_workspace_bytes": (_i64, [_i64, _i64, _i64, _i32]),
    "gqs_fp8_product": (_i32, [_vp, _vp, _i64, _vp, _vp, _i64, _i64, _i32, _vp, _i32, _vp, _i32,
                               _vp, _i64, _vp]),
    "gqs_fp8_linear_workspace_bytes": (_i64, [_i64, _i64, _i64, _i32]),
    "gqs_fp8_linear": (_i32, [_vp, _i32, _i64, _i64, _i64, _i32, _u64, _vp, _vp, _i64, _i32, _vp,
                              _i32, _vp, _vp, _i64, _vp]),
    "gqs_adamw": (_i32, [_vp, _i64, _i32, _i32, _args, _vp, _i64, _vp]),
    "gqs_moment8_restore": (_i32, [_vp, _vp, _i64, _i32, _i32, _vp, _vp]),
    "gqs_grad_norm_workspace_bytes": (_i64, [_vp, _i64]),
    "gqs_grad_norm": (_i32, [_vp, _i64, _i32, _f64, _vp, _vp, _vp, _i64, _vp]),
    "gqs_last_error": (ctypes.c_char_p, []),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libgq_step.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def check(status: int):
    if status != 0:
        raise GQError(status, lib().gqs_last_error().decode())
