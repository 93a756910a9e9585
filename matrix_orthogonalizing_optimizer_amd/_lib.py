"""ctypes binding of libmuon.so (the C ABI in include/muon.h).

Argument marshalling only: every step of the optimizer runs in the HIP
library.  Importing works without a GPU; there is no fallback of any kind --
if the library is not built, loading raises.
"""

from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmuon.so")

MO_OK, MO_EINVAL, MO_EUNSUPPORTED, MO_EWORKSPACE, MO_EHIP = 0, -1, -2, -3, -4
MO_F32, MO_BF16 = 0, 1
MO_SCALE_SHAPE, MO_SCALE_HIDDEN, MO_SCALE_UPDATE_NORM = 0, 1, 2
(MO_K_MOMENTUM, MO_K_NORM, MO_K_GRAM, MO_K_POLY, MO_K_UPDATE, MO_K_APPLY,
 MO_K_APPLY_X0, MO_K_RMS, MO_K_ADAMW, MO_K_SVD_GRAM, MO_K_SVD_REDUCE,
 MO_K_SVD_COLUMN, MO_K_SVD_EIG, MO_K_SVD_PANEL, MO_K_MX4_QUANT, MO_K_MX4_DEQUANT,
 MO_K_MX4_MATMUL, MO_K_LOGPROBS, MO_K_DISTILL, MO_K_FP8_QUANT, MO_K_FP8_DEQUANT,
 MO_K_FP8_MATMUL, MO_K_LINEAR_CE, MO_K_BALANCE) = range(24)
MO_MAX_TOP = 128
KERNEL_CLASS_NAMES = ["momentum", "norm", "gram", "poly", "update", "apply",
                      "apply_x0", "rms", "adamw", "svd_gram", "svd_reduce",
                      "svd_column", "svd_eig", "svd_panel", "mx4_quant", "mx4_dequant",
                      "mx4_matmul", "logprobs", "distill", "fp8_quant", "fp8_dequant",
                      "fp8_matmul", "linear_ce", "balance"]

STATUS_NAMES = {MO_OK: "MO_OK", MO_EINVAL: "MO_EINVAL",
                MO_EUNSUPPORTED: "MO_EUNSUPPORTED",
                MO_EWORKSPACE: "MO_EWORKSPACE", MO_EHIP: "MO_EHIP"}


class MoTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("state0", ctypes.c_void_p), ("state1", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class MoMatrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class MoMx4Image(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class MoMx4Item(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("codes_t", ctypes.c_void_p), ("scales_t", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64)]


class MoFp8Image(ctypes.Structure):
    _fields_ = MoMx4Image._fields_


class MoFp8Item(ctypes.Structure):
    _fields_ = MoMx4Item._fields_


class MuonError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


_c = ctypes
_P = _c.c_void_p
_SIGS = {
    "mo_abi_version": (_c.c_int, []),
    "mo_last_error": (_c.c_char_p, []),
    "mo_muon_workspace_size": (_c.c_int, [_c.POINTER(MoTensor), _c.c_int64, _c.c_int,
                                          _c.POINTER(_c.c_size_t), _c.POINTER(_c.c_size_t)]),
    "mo_muon_step": (_c.c_int, [_c.POINTER(MoTensor), _c.c_int64, _c.c_int, _c.c_int, _c.c_int,
                                _c.c_float, _c.c_float, _c.c_float, _c.c_int, _c.c_int,
                                _c.POINTER(_c.c_float), _c.c_float, _c.c_float,
                                _P, _P, _c.c_size_t, _P]),
    "mo_muon_step_noalloc": (_c.c_int, [_c.POINTER(MoTensor), _c.c_int64, _c.c_int, _c.c_int, _c.c_int,
                                        _c.c_float, _c.c_float, _c.c_float, _c.c_int, _c.c_int,
                                        _c.POINTER(_c.c_float), _c.c_float, _c.c_float, _P, _P]),
    "mo_muon_plan_create": (_c.c_int, [_c.POINTER(MoTensor), _c.c_int64, _c.c_int, _c.c_int,
                                       _c.c_int, _c.POINTER(_P)]),
    "mo_muon_plan_workspace_size": (_c.c_int, [_P, _c.POINTER(_c.c_size_t),
                                               _c.POINTER(_c.c_size_t)]),
    "mo_muon_plan_step": (_c.c_int, [_P, _c.c_float, _c.c_float, _c.c_float, _c.c_int, _c.c_int,
                                     _c.POINTER(_c.c_float), _c.c_float, _c.c_float,
                                     _P, _P, _c.c_size_t, _P]),
    "mo_muon_plan_set_scaling": (_c.c_int, [_P, _c.c_int, _c.c_float]),
    "mo_muon_plan_set_grads": (_c.c_int, [_P, _c.POINTER(_P), _c.c_int64, _P]),
    "mo_muon_plan_destroy": (_c.c_int, [_P]),
    "mo_adamw_step": (_c.c_int, [_c.POINTER(MoTensor), _c.c_int64, _c.c_int, _c.c_float,
                                 _c.c_float, _c.c_double, _c.c_double, _c.c_float, _c.c_int64, _P]),
    "mo_newton_schulz_workspace_size": (_c.c_int, [_c.c_int64, _c.c_int64, _c.c_int64, _c.c_int,
                                                   _c.POINTER(_c.c_size_t)]),
    "mo_newton_schulz": (_c.c_int, [_P, _P, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int, _c.c_int,
                                    _c.POINTER(_c.c_float), _c.c_float, _P, _c.c_size_t, _P]),
    "mo_svd_entropy_workspace_size": (_c.c_int, [_c.POINTER(MoMatrix), _c.c_int64,
                                                 _c.POINTER(_c.c_size_t), _c.POINTER(_c.c_size_t)]),
    "mo_svd_entropy": (_c.c_int, [_c.POINTER(MoMatrix), _c.c_int64, _c.c_int, _P, _P, _P,
                                  _c.c_size_t, _P]),
    "mo_mx4_image_size": (_c.c_int, [_c.c_int64, _c.c_int64, _c.POINTER(_c.c_size_t),
                                     _c.POINTER(_c.c_size_t)]),
    "mo_mx4_quantize": (_c.c_int, [_c.POINTER(MoMx4Item), _c.c_int64, _c.c_int, _P]),
    "mo_mx4_dequantize": (_c.c_int, [_c.POINTER(MoMx4Image), _c.POINTER(_P), _c.c_int64, _c.c_int, _P]),
    "mo_mx4_matmul": (_c.c_int, [_c.POINTER(MoMx4Image), _c.POINTER(MoMx4Image), _P, _c.c_int,
                                 _c.c_int64, _c.c_int, _P]),
    "mo_token_logprobs_workspace_size": (_c.c_int, [_c.c_int64, _c.c_int64, _c.c_int,
                                                    _c.POINTER(_c.c_size_t)]),
    "mo_distill_loss_workspace_size": (_c.c_int, [_c.c_int64, _c.c_int64, _c.c_int,
                                                  _c.POINTER(_c.c_size_t)]),
    "mo_token_logprobs": (_c.c_int, [_P, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _P, _c.c_float,
                                     _P, _P, _c.c_int, _P, _P, _P, _c.c_size_t, _P]),
    "mo_distill_loss": (_c.c_int, [_P, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _P, _P, _c.c_int,
                                   _c.c_float, _P, _P, _P, _c.c_int64, _P, _c.c_size_t, _P]),
    "mo_fp8_image_size": (_c.c_int, [_c.c_int64, _c.c_int64, _c.POINTER(_c.c_size_t),
                                     _c.POINTER(_c.c_size_t)]),
    # items, images and destinations as any array of 64-bit values: filling a flat one costs a
    # third of setting fields
    "mo_fp8_quantize": (_c.c_int, [_P, _c.c_int64, _c.c_int, _c.c_int, _P]),
    "mo_fp8_dequantize": (_c.c_int, [_P, _P, _c.c_int64, _c.c_int, _P]),
    "mo_fp8_matmul": (_c.c_int, [_P, _P, _P, _c.c_int, _c.c_int64, _c.c_int, _P]),
    "mo_linear_ce_workspace_size": (_c.c_int, [_c.c_int64, _c.c_int64, _c.c_int64, _c.c_int, _c.c_int,
                                               _c.c_int, _c.c_int, _c.POINTER(_c.c_size_t)]),
    "mo_linear_ce": (_c.c_int, [_P, _c.c_int, _c.c_int64, _P, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64,
                                _c.c_int64, _P, _P, _P, _P, _c.c_int64, _P, _c.c_int, _c.c_int64, _c.c_int,
                                _P, _c.c_size_t, _P]),
    "mo_balance_loss_workspace_size": (_c.c_int, [_c.c_int64, _c.c_int64, _c.POINTER(_c.c_size_t)]),
    "mo_balance_loss": (_c.c_int, [_P, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _P, _c.c_int64,
                                   _c.c_float, _P, _P, _P, _P, _c.c_int64, _c.c_int, _P, _c.c_size_t, _P]),
    "mo_profile_enable": (_c.c_int, [_c.c_uint]),
    "mo_profile_read": (_c.c_int, [_c.c_int, _c.POINTER(_c.c_int64), _c.POINTER(_c.c_double),
                                   _c.POINTER(_c.c_double)]),
    "mo_profile_reset": (_c.c_int, []),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m matrix_orthogonalizing_optimizer_amd.build` "
                "(there is no non-HIP fallback)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def last_error() -> str:
    msg = lib().mo_last_error()
    return msg.decode() if msg else ""


def check(code: int) -> None:
    if code != MO_OK:
        raise MuonError(code, last_error())
