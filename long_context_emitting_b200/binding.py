"""ctypes binding of libkascade.so: the C entry points under the same names.

Only argument marshalling lives here.  Every entry point takes raw device
pointers (ints) and sizes, exactly as declared in include/kascade.h.  Loading
fails loudly when the library has not been built: there is no fallback.
"""
from __future__ import annotations

import ctypes
import operator
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkascade.so")

KASCADE_OK = 0
STATIC_SCRATCH_BYTES = 16 * 1024 * 1024  # KASCADE_STATIC_SCRATCH_BYTES in include/kascade.h
Q4_ROW_BYTES = 160  # KASCADE_Q4_ROW_BYTES: one token of one key head, K and V
STATUS_NAMES = {
    0: "KASCADE_OK",
    1: "KASCADE_ERR_INVALID_ARG",
    2: "KASCADE_ERR_UNSUPPORTED_SHAPE",
    3: "KASCADE_ERR_WORKSPACE_TOO_SMALL",
    4: "KASCADE_ERR_CUDA",
    5: "KASCADE_ERR_BAD_INDEX",
    6: "KASCADE_ERR_NONFINITE",
    7: "KASCADE_ERR_TIMEOUT",
}
KASCADE_ERR_TIMEOUT = 7

# Every symbol the header declares (checked by the CPU tests).
EXPORTS = (
    "kascade_k_for_len",
    "kascade_decode_anchor_workspace_bytes",
    "kascade_decode_anchor",
    "kascade_decode_anchor_static_ws",
    "kascade_topk_workspace_bytes",
    "kascade_topk",
    "kascade_decode_reuse_workspace_bytes",
    "kascade_decode_reuse",
    "kascade_prefill_anchor_workspace_bytes",
    "kascade_prefill_anchor",
    "kascade_prefill_reuse_workspace_bytes",
    "kascade_prefill_reuse",
    "kascade_decode_anchor_f16",
    "kascade_decode_reuse_f16",
    "kascade_prefill_anchor_f16",
    "kascade_prefill_reuse_f16",
    "kascade_decode_anchor_paged",
    "kascade_decode_reuse_paged",
    "kascade_decode_anchor_paged_f16",
    "kascade_decode_reuse_paged_f16",
    "kascade_qk_norm_rope",
    "kascade_qk_norm_rope_f16",
    "kascade_kv_write_paged_q4",
    "kascade_kv_write_paged_q4_f16",
    "kascade_kv_read_paged_q4",
    "kascade_kv_read_paged_q4_f16",
    "kascade_decode_anchor_paged_q4_workspace_bytes",
    "kascade_decode_anchor_paged_q4",
    "kascade_decode_anchor_paged_q4_f16",
    "kascade_decode_reuse_paged_q4",
    "kascade_decode_reuse_paged_q4_f16",
    "kascade_similarity_rows",
    "kascade_similarity_mean_workspace_bytes",
    "kascade_similarity_mean",
    "kascade_head_remap_workspace_bytes",
    "kascade_head_remap",
    "kascade_select_anchors",
    "kascade_get_device_status",
    "kascade_status_string",
    "kascade_selftest_wait_timeout",
    "kascade_selftest_anchor_q4_gives_up",
)


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("d", ctypes.c_int32)]


class Strides(ctypes.Structure):
    """Element strides between sequences, tokens and heads (kascade_strides)."""
    _fields_ = [("b", ctypes.c_int64), ("n", ctypes.c_int64), ("h", ctypes.c_int64)]


class KascadeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float

_SIGNATURES = {
    "kascade_k_for_len": (_I32, [_I32]),
    "kascade_decode_anchor_workspace_bytes": (_SZ, [Shape, _I32]),
    "kascade_decode_anchor": (ctypes.c_int, [Shape, _P, _P, _P, _P, _P, _I32, _F, _P, _P, _P, _I64,
                                             _P, _SZ, _P]),
    "kascade_decode_anchor_static_ws": (ctypes.c_int, [Shape, _P, _P, _P, _P, _P, _I32, _F, _P, _P,
                                                       _P, _I64, _P]),
    "kascade_topk_workspace_bytes": (_SZ, [_I32, _I64]),
    "kascade_topk": (ctypes.c_int, [_P, _I32, _I64, _P, _P, _I32, _P, _P, _SZ, _P]),
    "kascade_decode_reuse_workspace_bytes": (_SZ, [Shape, _I32]),
    "kascade_decode_reuse": (ctypes.c_int, [Shape, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _F, _P,
                                            _P, _P, _SZ, _P]),
    "kascade_prefill_anchor_workspace_bytes": (_SZ, [Shape, _I32]),
    "kascade_prefill_anchor": (ctypes.c_int, [Shape, _I32, _P, _P, _P, _F, _P, _P, _P, _P, _SZ,
                                              _P]),
    "kascade_prefill_reuse_workspace_bytes": (_SZ, [Shape, _I32, _I32]),
    "kascade_prefill_reuse": (ctypes.c_int, [Shape, _I32, _P, _P, _P, _P, _P, _I32, _P, _F, _P, _P,
                                             _P, _SZ, _P]),
    "kascade_decode_anchor_paged": (ctypes.c_int, [Shape, _P, _P, _P, _I32, _P, _I32, _I32, _P, _I32,
                                                   _F, _P, _P, _P, _I64, _P, _SZ, _P]),
    "kascade_decode_reuse_paged": (ctypes.c_int, [Shape, _P, _P, _P, _I32, _P, _I32, _I32, _P, _P,
                                                  _P, _I32, _P, _F, _P, _P, _P, _SZ, _P]),
    "kascade_qk_norm_rope": (ctypes.c_int, [Shape, _I32, _P, Strides, _P, Strides, _P, _P, _P, _P, _F, _I32,
                                            _P, Strides, _P, Strides, _P]),
    "kascade_kv_write_paged_q4": (ctypes.c_int, [Shape, _I32, _P, Strides, _P, Strides, _P, _I32, _P, _I32, _I32,
                                                 _P, _P, _P]),
    "kascade_kv_read_paged_q4": (ctypes.c_int, [Shape, _I32, _P, _I32, _P, _I32, _I32, _P, _P, _P, _P, _P]),
    "kascade_decode_anchor_paged_q4_workspace_bytes": (_SZ, [Shape, _I32]),
    "kascade_decode_anchor_paged_q4": (ctypes.c_int, [Shape, _P, _P, _I32, _P, _I32, _I32, _P, _I32, _F, _P, _P,
                                                      _P, _I64, _P, _SZ, _P]),
    "kascade_decode_reuse_paged_q4": (ctypes.c_int, [Shape, _P, _P, _I32, _P, _I32, _I32, _P, _P, _P, _I32, _P,
                                                     _F, _P, _P, _P]),
    "kascade_similarity_rows": (ctypes.c_int, [_P, _I32, _I64, _P, _P, _P, _P, _I32, _I32, _P, _P,
                                               _P, _P]),
    "kascade_similarity_mean_workspace_bytes": (_SZ, [_I32]),
    "kascade_similarity_mean": (ctypes.c_int, [_P, _I32, _I64, _P, _P, _P, _P, _I32, _P, _P, _SZ,
                                               _P]),
    "kascade_head_remap_workspace_bytes": (_SZ, [_I32, _I32]),
    "kascade_head_remap": (ctypes.c_int, [_P, _I32, _I32, _I64, _P, _P, _P, _P, _I32, _P, _P, _P,
                                          _SZ, _P]),
    "kascade_select_anchors": (ctypes.c_int, [_P, _I32, _I32, _P, _P]),
    "kascade_get_device_status": (ctypes.c_int, [_P]),
    "kascade_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "kascade_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_int32, _P]),
    "kascade_selftest_anchor_q4_gives_up": (ctypes.c_int, [_I32, Shape, _P, _P, _I32, _P, _I32, _I32, _P, _I32, _F, _P,
                                                           _P, _P, _I64, _P, _SZ, _P]),
}
# fp16 variants take the same arguments as their bfloat16 counterparts
for _name in ("kascade_decode_anchor", "kascade_decode_reuse", "kascade_prefill_anchor",
              "kascade_prefill_reuse", "kascade_decode_anchor_paged", "kascade_decode_reuse_paged",
              "kascade_qk_norm_rope", "kascade_kv_write_paged_q4", "kascade_kv_read_paged_q4",
              "kascade_decode_anchor_paged_q4", "kascade_decode_reuse_paged_q4"):
    _SIGNATURES[_name + "_f16"] = _SIGNATURES[_name]

_lib = None


# What _hostcall calls, in its order: host_<name> of the library object takes the entry point's
# arguments as plain numbers (half precision 0 or 1 first, structures by their fields).  Where that
# module has not been built (it needs Python's headers), the same calls go through ctypes.
HOSTCALLS = {
    "norm_rope": "kascade_qk_norm_rope",
    "kv_write": "kascade_kv_write_paged_q4",
    "kv_read": "kascade_kv_read_paged_q4",
    "decode_anchor": "kascade_decode_anchor_paged_q4",
    "decode_reuse": "kascade_decode_reuse_paged_q4",
}


def ctypes_hostcall(lib: ctypes.CDLL, name: str):
    """host_<name> through ctypes: the same arguments, refusals and status, 2 us slower."""
    fns = [getattr(lib, HOSTCALLS[name] + sfx) for sfx in ("", "_f16")]
    types = _SIGNATURES[HOSTCALLS[name]][1]
    plain = [f for t in types for f in ([x for _, x in t._fields_] if issubclass(t, ctypes.Structure) else [t])]

    def number(t, x):
        if t is _F:
            return float(x)
        x = None if x is None else operator.index(x)
        if x is None:
            return x if t is _P else 0
        bits = 8 * ctypes.sizeof(_I32 if t is _I32 else _I64)
        if not -(1 << bits - 1) <= x < 1 << bits - 1:
            raise OverflowError(f"{x} does not fit {bits} bits")
        return x

    def call(*args):
        if len(args) != 1 + len(plain):
            raise TypeError(f"{len(args)} arguments, not {1 + len(plain)}")
        half = number(_I32, args[0])
        given = iter([number(t, x) for t, x in zip(plain, args[1:])])
        return fns[half != 0](*[t(*[next(given) for _ in t._fields_]) if issubclass(t, ctypes.Structure) else next(given)
                                for t in types])
    return call


def _bind_hostcalls(lib: ctypes.CDLL) -> None:
    try:
        from . import _hostcall
    except ImportError:
        for name in HOSTCALLS:
            setattr(lib, "host_" + name, ctypes_hostcall(lib, name))
        return
    _hostcall.bind(*(ctypes.cast(getattr(lib, name + sfx), ctypes.c_void_p).value
                     for name in HOSTCALLS.values() for sfx in ("", "_f16")))
    for name in HOSTCALLS:
        setattr(lib, "host_" + name, getattr(_hostcall, name))


def load() -> ctypes.CDLL:
    """Load libkascade.so (built in-tree) and declare every signature."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m long_context_emitting_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _bind_hostcalls(lib)
    _lib = lib
    return lib


def check(status: int, where: str) -> None:
    if status != KASCADE_OK:
        raise KascadeError(status, where)
