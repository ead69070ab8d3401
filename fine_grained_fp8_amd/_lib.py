"""ctypes loader for libfp8bs.so and the C-ABI declarations.

The library is the only implementation: if it is not built, loading raises.
There is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8bs.so")

STATUS = {
    0: "FP8_OK", 1: "FP8_ERR_NULL", 2: "FP8_ERR_SHAPE", 3: "FP8_ERR_LD", 4: "FP8_ERR_ALIGN",
    5: "FP8_ERR_UNSUPPORTED", 6: "FP8_ERR_DEVICE", 7: "FP8_ERR_LAUNCH", 8: "FP8_ERR_ALIAS",
}
TILE_ROW, TILE_COL, TILE_COL_TILED = 0, 1, 2
LAYOUT = {"fprop": 0, "dgrad": 1, "wgrad": 2, "dgrad_t": 3, "fprop_tiled": 4, "dgrad_t_tiled": 5, "wgrad_tiled": 6}
OUT_BF16, OUT_FP32 = 0, 1
MOE_GATE = {"softmax": 0, "sigmoid": 1}
ACTIVATION = {"silu": 0, "gelu": 1}
HEAD_NORM = {None: 0, "rms": 1, "layer": 2}

# name -> (restype, argtypes); mirrors include/fp8bs.h
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_F = ctypes.c_float


class Heads(ctypes.Structure):
    """fp8_heads"""
    _fields_ = [("x", _P), ("heads", _I64), ("ld_token", _I64), ("ld_head", _I64), ("weight", _P), ("y", _P),
                ("ldy_token", _I64), ("ldy_head", _I64)]


class HeadsGrad(ctypes.Structure):
    """fp8_heads_grad"""
    _fields_ = [("x", _P), ("heads", _I64), ("ld_token", _I64), ("ld_head", _I64), ("weight", _P), ("dy", _P),
                ("lddy_token", _I64), ("lddy_head", _I64), ("dx", _P), ("lddx_token", _I64), ("lddx_head", _I64),
                ("dweight", _P)]


_HEAD_ARGS = [ctypes.c_int, ctypes.c_int, _F, _I64, _P, _I32, _I32, ctypes.POINTER(_I64), _P, _I32]
SIGNATURES = {
    "fp8_quant_act_1x128": (ctypes.c_int, [_P, _I64, _I64, _I64, ctypes.c_int, _P, _I64, _P, _I64,
                                           _P, _P, _P, _P]),
    "fp8_quant_act_dual": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                                          _P]),
    "fp8_quant_act_dual_tiled": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _P, _I64,
                                                _P]),
    "fp8_quant_weight_128x128": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _P]),
    "fp8_block_gemm": (ctypes.c_int, [ctypes.c_int, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _P,
                                      _I64, _P, ctypes.c_int, _I64, _P]),
    "fp8_block_gemm_noalloc": (ctypes.c_int, [ctypes.c_int, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64,
                                              _P, _I64, _P, ctypes.c_int, _I64, _P]),
    "fp8_quant_weight_128x128_tiled": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _P, _I64, _P]),
    "fp8_block_gemm_grouped_tiled": (ctypes.c_int, [_I32, _P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P,
                                                    _P, _P, ctypes.c_int, _I64, _P]),
    "fp8_block_gemm_fused_quant": (ctypes.c_int, [_I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _P,
                                                  ctypes.c_int, _I64, _P, _I64, _P, _I64, _P]),
    "fp8_block_gemm_grouped": (ctypes.c_int, [_I32, _P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64,
                                              _P, _P, ctypes.c_int, _I64, _P]),
    "fp8_amax_history_update": (ctypes.c_int, [_P, _P, _I64, _F, ctypes.c_int, _P, _P]),
    "fp8_cast_e4m3": (ctypes.c_int, [_P, _I64, _P, _P]),
    "fp8_quant_act_tiles": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _I32, _P, _I64, _P, _I64, _P, _P]),
    "fp8_gemm_promotion": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _I64, _I64, _P, _I64, _P]),
    "fp8_probe_mfma": (ctypes.c_int, [_I64, ctypes.c_int32, ctypes.c_int32, _P, _P, _P]),
    "fp8_probe_recip_online": (ctypes.c_int, [_P, _P, _I64, _P]),
    "fp8_probe_gemm_split": (ctypes.c_int, [_I64, _I64, _P, _P, _P]),
    "fp8_pack_tokens": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P]),
    "fp8_unpack_tokens": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P]),
    "fp8_dequant_tokens": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _P]),
    "fp8_layer_norm": (ctypes.c_int, [_P, _I64, _I64, _I64, ctypes.c_int, _P, _P, ctypes.c_int, _F, _P, _I64, _P,
                                      _P, _P, _I64, _P, _I64, _P]),
    "fp8_layer_norm_backward": (ctypes.c_int, [_P, _I64, _P, _I64, _I64, _I64, ctypes.c_int, _P, _P, _P,
                                               ctypes.c_int, _P, _I64, _P, _P, _P, _I64, _P]),
    "fp8_layer_norm_backward_workspace": (_I64, [_I64, _I64]),
    "fp8_moe_few_tokens": (ctypes.c_int, [_I64, _I64, _I64, _I32, _I32, _I32, _I32, _P, _I64, _P, _I64, _P,
                                          ctypes.c_int, ctypes.c_int, _F, _P, _P, _P, _P, _P, ctypes.c_int, _I64,
                                          _P, _P, _P, _I64, _P]),
    "fp8_moe_few_tokens_workspace": (_I64, [_I64, _I64, _I64, _I32, _I32, _I32]),
    "fp8_adapter_linear": (ctypes.c_int, [_I64, _I64, _I64, _I32, _I32, _P, _I64, _P, _P, _I64, _P, _P, _P, _P,
                                          _P, ctypes.c_int, _I64, _P, _I64, _P]),
    "fp8_adapter_linear_workspace": (_I64, [_I64, _I64, _I64, _I32, _I32]),
    "fp8_block_gemm_gated": (ctypes.c_int, [_I64, _I64, _I64, _P, _I64, _P, _I64, _P, _P, _I64, ctypes.c_int, _P,
                                            ctypes.c_int, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P]),
    "fp8_block_gemm_gated_workspace": (_I64, [_I64, _I64, _I64, ctypes.c_int, _I32]),
    "fp8_gated_backward": (ctypes.c_int, [_I64, _I64, _P, _I64, _P, _I64, ctypes.c_int, _P, _I64, _P, _I64, _P, _I64,
                                          _P, _I64, _P, _I64, _P, _P, _I64, _P]),
    "fp8_quant_act_cols": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _I64, _P]),
    "fp8_head_norm_rotary": (ctypes.c_int, [_I64, _I64, ctypes.c_int, ctypes.POINTER(Heads), ctypes.POINTER(Heads),
                                            *_HEAD_ARGS, _P]),
    "fp8_head_norm_rotary_backward": (ctypes.c_int, [_I64, _I64, ctypes.c_int, ctypes.POINTER(HeadsGrad),
                                                     ctypes.POINTER(HeadsGrad), *_HEAD_ARGS, _P, _I64, _P]),
    "fp8_head_norm_rotary_backward_workspace": (_I64, [_I64, _I64, _I64, _I64]),
    "fp8_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "fp8_abi_version": (ctypes.c_int, []),
}

# the entry points of api_layers.cpp and of api_blocks.cpp; the others are api.cpp's
LAYER_ENTRIES = {n for n in SIGNATURES if n.startswith(("fp8_layer_norm", "fp8_moe_", "fp8_adapter_"))}
BLOCK_ENTRIES = {n for n in SIGNATURES
                 if n.startswith(("fp8_block_gemm_gated", "fp8_gated_", "fp8_quant_act_cols", "fp8_head_"))}
_PARTS = (LAYER_ENTRIES, BLOCK_ENTRIES, set(SIGNATURES) - LAYER_ENTRIES - BLOCK_ENTRIES)

_lib = None
_lock = threading.Lock()


class FP8Error(RuntimeError):
    """A non-OK status from libfp8bs."""

    def __init__(self, fn: str, status: int):
        self.status = status
        msg = STATUS.get(status, str(status))
        detail = ""
        if _lib is not None:
            try:
                detail = _lib.fp8_status_string(status).decode()
            except Exception:  # pragma: no cover
                pass
        super().__init__(f"{fn}: {msg} ({detail})")


def load_library(path: str | None = None):
    """Load libfp8bs.so (once).  Raises OSError/RuntimeError if it is absent.

    A library named by `path` may be a host-only build of one source file of the
    ABI: it has to have all of that file's entry points, and of another's all or
    none.  The built library has to have them all."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"{p} is not built; run `python -m fine_grained_fp8_amd.build` "
                "(there is no CPU fallback)")
        lib = ctypes.CDLL(p)
        missing = {n for n in SIGNATURES if not hasattr(lib, n)}
        whole = all(part <= missing or not part & missing for part in _PARTS)
        if missing and (path is None or not whole or len(missing) == len(SIGNATURES)):
            raise RuntimeError(f"{p} lacks {', '.join(sorted(missing))}: build it again")
        for name, (res, args) in SIGNATURES.items():
            if name in missing:
                continue
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def check(fn: str, status: int) -> None:
    if status != 0:
        raise FP8Error(fn, status)
