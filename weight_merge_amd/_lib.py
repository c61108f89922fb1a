"""ctypes declarations of libadafuse's C ABI (include/adafuse.h)."""
from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libadafuse.so")

ADA_OK, ADA_EINVAL, ADA_ESHAPE, ADA_EDTYPE, ADA_EALIGN, ADA_EHIP, ADA_ENOMEM = 0, -1, -2, -3, -4, -5, -6
ADA_F32, ADA_BF16 = 0, 1
ADA_ACT_NONE, ADA_ACT_RELU, ADA_ACT_SILU, ADA_ACT_GELU, ADA_ACT_GELU_TANH = 0, 1, 2, 3, 4

c_void_p = ctypes.c_void_p
c_int32 = ctypes.c_int32
c_int64 = ctypes.c_int64
c_float = ctypes.c_float


class AdaProj(ctypes.Structure):
    _fields_ = [
        ("w", c_void_p),
        ("w_out", c_void_p),
        ("a", c_void_p),
        ("b", c_void_p),
        ("d_out", c_int32),
        ("d_in", c_int32),
        ("ld_w", c_int64),
    ]


class AdaLoraProj(ctypes.Structure):
    _fields_ = [
        ("w", c_void_p),
        ("a", c_void_p),
        ("b", c_void_p),
        ("x", c_void_p),
        ("y", c_void_p),
        ("d_out", c_int32),
        ("d_in", c_int32),
        ("ld_w", c_int64),
    ]


class AdaGemvProj(ctypes.Structure):
    _fields_ = [
        ("w", c_void_p),
        ("x", c_void_p),
        ("y", c_void_p),
        ("d_out", c_int32),
        ("d_in", c_int32),
        ("ld_w", c_int64),
    ]


class AdaLinearArgs(ctypes.Structure):
    _fields_ = (
        [(n, c_void_p) for n in ("x", "w", "bias", "residual", "y", "pre")]
        + [(n, c_int64) for n in ("ld_x", "ld_w", "ld_res", "ld_y", "ld_pre", "rows")]
        + [("d_out", c_int32), ("d_in", c_int32)]
    )


class AdaLinearGradArgs(ctypes.Structure):
    _fields_ = (
        [(n, c_void_p) for n in ("dy", "x", "w", "pre", "dx", "dw", "dbias")]
        + [(n, c_int64) for n in ("ld_dy", "ld_x", "ld_w", "ld_pre", "ld_dx", "ld_dw", "rows")]
        + [("d_out", c_int32), ("d_in", c_int32)]
    )


class AdaGluArgs(ctypes.Structure):
    _fields_ = (
        [(n, c_void_p) for n in ("x", "w_gate", "w_up", "bias_gate", "bias_up", "y", "gate_pre", "up_pre")]
        + [(n, c_int64) for n in ("ld_x", "ld_w_gate", "ld_w_up", "ld_y", "ld_gate_pre", "ld_up_pre", "rows")]
        + [("d_out", c_int32), ("d_in", c_int32)]
    )


class AdaGluGradArgs(ctypes.Structure):
    _fields_ = (
        [(n, c_void_p) for n in ("dy", "x", "w_gate", "w_up", "gate_pre", "up_pre", "dx", "dw_gate", "dw_up", "dbias_gate", "dbias_up")]
        + [(n, c_int64) for n in ("ld_dy", "ld_x", "ld_w_gate", "ld_w_up", "ld_gate_pre", "ld_up_pre", "ld_dx", "ld_dw_gate", "ld_dw_up", "rows")]
        + [("d_out", c_int32), ("d_in", c_int32)]
    )


_SIGNATURES = {
    "ada_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ada_model_create": (ctypes.c_int, [ctypes.POINTER(AdaProj), c_int32, c_int32, c_int32, c_int32,
                                        c_void_p, ctypes.POINTER(c_void_p)]),
    "ada_model_destroy": (None, [c_void_p]),
    "ada_model_tiles": (c_int64, [c_void_p]),
    "ada_model_device_bytes": (c_int64, [c_void_p]),
    "ada_pregate": (ctypes.c_int, [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32, c_int32,
                                   c_void_p, c_void_p, c_void_p]),
    "ada_merge": (ctypes.c_int, [c_void_p, c_void_p, c_void_p, c_int32, c_float, c_void_p]),
    "ada_unmerge": (ctypes.c_int, [c_void_p, c_void_p, c_void_p, c_int32, c_float, c_void_p]),
    "ada_switch": (ctypes.c_int, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32,
                                  c_float, c_void_p]),
    "ada_decode_gemv": (ctypes.c_int, [c_void_p, c_int32, c_int32, c_int64, c_void_p, c_void_p, c_int32,
                                       c_void_p]),
    "ada_decode_gemv_layer": (ctypes.c_int, [ctypes.POINTER(AdaGemvProj), c_int32, c_int32, c_void_p]),
    "ada_lora_apply": (ctypes.c_int, [c_void_p, c_int32, c_int32, c_int64, c_void_p, c_void_p, c_int32,
                                      c_int32, c_void_p, c_void_p, c_int32, c_float, c_void_p, c_void_p,
                                      c_void_p, c_int64, c_int32, c_void_p]),
    "ada_lora_layer": (ctypes.c_int, [ctypes.POINTER(AdaLoraProj), c_int32, c_int32, c_int32, c_void_p, c_void_p,
                                      c_int32, c_float, c_void_p, c_int64, c_int32, c_void_p]),
    "ada_lora_layer_static": (ctypes.c_int, [ctypes.POINTER(AdaLoraProj), c_int32, c_int32, c_int32, c_void_p,
                                             c_void_p, c_int32, c_float, c_int32, c_void_p]),
    "ada_lora_batch": (ctypes.c_int, [ctypes.POINTER(AdaLoraProj), c_int32, c_int32, c_int32, c_int32, c_void_p,
                                      c_void_p, c_int32, c_float, c_void_p, c_int64, c_int32, c_void_p]),
    "ada_linear": (ctypes.c_int, [ctypes.POINTER(AdaLinearArgs), c_int32, c_int32, c_void_p, c_int64, c_void_p]),
    "ada_linear_workspace": (c_int64, [c_int64, c_int32, c_int32, c_int32]),
    "ada_linear_backward": (ctypes.c_int, [ctypes.POINTER(AdaLinearGradArgs), c_int32, c_int32, c_void_p, c_int64,
                                           c_void_p]),
    "ada_linear_backward_workspace": (c_int64, [c_int64, c_int32, c_int32, c_int32, c_int32]),
    "ada_glu": (ctypes.c_int, [ctypes.POINTER(AdaGluArgs), c_int32, c_int32, c_void_p, c_int64, c_void_p]),
    "ada_glu_workspace": (c_int64, [c_int64, c_int32, c_int32, c_int32]),
    "ada_glu_backward": (ctypes.c_int, [ctypes.POINTER(AdaGluGradArgs), c_int32, c_int32, c_void_p, c_int64, c_void_p]),
    "ada_glu_backward_workspace": (c_int64, [c_int64, c_int32, c_int32, c_int32, c_int32]),
}

_lib = None


class LibraryMissing(RuntimeError):
    pass


def load():
    """Load libadafuse.so (built in-tree).  There is no fallback: a missing library
    is an error."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise LibraryMissing(
                f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
                "or `python weight_merge_amd/build.py` first")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def declared_functions(header: str) -> list[str]:
    """Function names a C header declares (for the export check)."""
    import re

    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(ada_[a-z_]+)\s*\(", text)))
