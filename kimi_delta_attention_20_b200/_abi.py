"""ctypes mirror of include/kda.h. Argument marshalling only.

Loading fails loudly (ImportError) when libkda.so is missing: there is no
fallback implementation behind this binding.
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")

KDA_OK = 0
KDA_ERR_INVALID_ARGUMENT = 1
KDA_ERR_UNSUPPORTED = 2
KDA_ERR_CUDA = 3
KDA_ERR_TIMEOUT = 4
KDA_ERR_WORKSPACE = 5

KDA_DTYPE_F32 = 0
KDA_DTYPE_BF16 = 1

KDA_GATE_LOG = 0
KDA_GATE_SOFTPLUS = 1
KDA_GATE_SAFE = 2

KDA_SCAN_GATE_LOG = 0
KDA_SCAN_GATE_SIGMOID = 1

KDA_DEBUG_STALL_FIRST_WAIT = 1

_vp = ctypes.c_void_p
_fp = ctypes.POINTER(ctypes.c_float)
_i32p = ctypes.POINTER(ctypes.c_int32)


class ChunkArgs(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
        ("Dk", ctypes.c_int), ("Dv", ctypes.c_int),
        ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp),
        ("o", _vp),
        ("scale", ctypes.c_float),
        ("initial_state", _vp), ("final_state", _vp),
        ("cu_seqlens", _vp), ("cu_seqlens_host", _vp),
        ("N", ctypes.c_int),
        ("use_qk_l2norm", ctypes.c_int),
        ("has_lower_bound", ctypes.c_int), ("lower_bound", ctypes.c_float),
        ("chunk_size", ctypes.c_int),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
        ("gate_mode", ctypes.c_int), ("A_log", _vp), ("dt_bias", _vp),
        ("beta_is_prob", ctypes.c_int),
        ("debug_flags", ctypes.c_uint),
    ]


class StepArgs(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("N", ctypes.c_int), ("H", ctypes.c_int), ("Dk", ctypes.c_int), ("Dv", ctypes.c_int),
        ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp),
        ("state", _vp), ("o", _vp),
        ("scale", ctypes.c_float),
        ("use_qk_l2norm", ctypes.c_int),
        ("has_lower_bound", ctypes.c_int), ("lower_bound", ctypes.c_float),
        ("gate_mode", ctypes.c_int), ("A_log", _vp), ("dt_bias", _vp),
        ("beta_is_prob", ctypes.c_int),
        ("state_out", _vp),
    ]


class TokenArgs(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("N", ctypes.c_int), ("H", ctypes.c_int), ("Dk", ctypes.c_int), ("Dv", ctypes.c_int),
        ("conv_kernel", ctypes.c_int),
        ("x", _vp), ("conv_w", _vp), ("conv_state", _vp), ("g", _vp), ("beta", _vp),
        ("state", _vp), ("g_out", _vp), ("norm_eps", ctypes.c_float), ("o", _vp),
        ("scale", ctypes.c_float),
        ("use_qk_l2norm", ctypes.c_int),
        ("has_lower_bound", ctypes.c_int), ("lower_bound", ctypes.c_float),
        ("gate_mode", ctypes.c_int), ("A_log", _vp), ("dt_bias", _vp),
        ("beta_is_prob", ctypes.c_int),
        ("state_out", _vp),
    ]


class BwdArgs(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
        ("Dk", ctypes.c_int), ("Dv", ctypes.c_int),
        ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp),
        ("dout", _vp),
        ("scale", ctypes.c_float),
        ("initial_state", _vp), ("dfinal_state", _vp),
        ("dq", _vp), ("dk", _vp), ("dv", _vp), ("dg", _vp), ("dbeta", _vp),
        ("dinitial_state", _vp),
        ("cu_seqlens", _vp), ("cu_seqlens_host", _vp),
        ("N", ctypes.c_int),
        ("use_qk_l2norm", ctypes.c_int),
        ("has_lower_bound", ctypes.c_int), ("lower_bound", ctypes.c_float),
        ("beta_is_prob", ctypes.c_int),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


_i, _ll, _f, _sz = ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t
_SPAN = [("cu_seqlens", _vp), ("cu_seqlens_host", _vp), ("N", _i)]
_SCRATCH = [("workspace", _vp), ("workspace_bytes", _sz)]


def _rows(*names):
    """Pointer and row stride of each of the named tensors."""
    return [f for n in names for f in ((n, _vp), (n + "_stride", _ll))]


class RMSNormArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("weight_dtype", _i), ("rows", _ll), ("heads", _i), ("D", _i), *_rows("x", "residual", "gate"),
                ("weight", _vp), ("eps", _f), ("y", _vp), ("residual_out", _vp), ("scales", _vp), ("group_size", _i),
                ("pow2_scales", _i)]


class RMSNormBwdArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("weight_dtype", _i), ("rows", _ll), ("heads", _i), ("D", _i),
                *_rows("x", "dy", "gate", "dresidual"), ("weight", _vp), ("eps", _f), ("dx", _vp), ("dgate", _vp),
                ("dweight", _vp), *_SCRATCH]


class ConvArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("B", _i), ("T", _i), ("C", _i), ("K", _i), *_rows("x"), ("conv_w", _vp),
                ("initial_state", _vp), ("final_state", _vp), ("y", _vp), *_SPAN]


class ConvStepArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("N", _i), ("C", _i), ("K", _i), *_rows("x"), ("conv_w", _vp), ("conv_state", _vp),
                ("y", _vp)]


class ConvBwdArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("B", _i), ("T", _i), ("C", _i), ("K", _i), *_rows("x", "dy"), ("conv_w", _vp),
                ("initial_state", _vp), ("dfinal_state", _vp), ("dx", _vp), ("dconv_w", _vp),
                ("dinitial_state", _vp), *_SPAN, *_SCRATCH]


class ScanArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("gate", _i), ("B", _i), ("T", _i), ("D", _i), *_rows("x", "g"), ("h", _vp),
                ("initial_state", _vp), ("final_state", _vp), *_SPAN, ("has_lower_bound", _i), ("lower_bound", _f),
                *_SCRATCH]


class ScanStepArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("gate", _i), ("N", _i), ("D", _i), *_rows("x", "g"), ("state", _vp),
                ("state_out", _vp), ("h", _vp), ("has_lower_bound", _i), ("lower_bound", _f)]


class ScanBwdArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("gate", _i), ("B", _i), ("T", _i), ("D", _i), *_rows("x", "g", "h", "dout"),
                ("initial_state", _vp), ("dfinal_state", _vp), ("dx", _vp), ("dg", _vp), ("dinitial_state", _vp),
                *_SPAN, ("has_lower_bound", _i), ("lower_bound", _f), *_SCRATCH]


# entry points of the operators around the state update: name -> argument struct
_LAYER = {
    "kda_rms_norm": RMSNormArgs, "kda_rms_norm_bwd": RMSNormBwdArgs, "kda_causal_conv": ConvArgs,
    "kda_causal_conv_step": ConvStepArgs, "kda_causal_conv_bwd": ConvBwdArgs, "kda_gated_scan": ScanArgs,
    "kda_gated_scan_step": ScanStepArgs, "kda_gated_scan_bwd": ScanBwdArgs,
}
_LAYER_SIZES = {
    "kda_rms_norm_bwd_workspace_size": RMSNormBwdArgs, "kda_causal_conv_bwd_workspace_size": ConvBwdArgs,
    "kda_gated_scan_workspace_size": ScanArgs, "kda_gated_scan_bwd_workspace_size": ScanBwdArgs,
}

_CODES = {_i: "i", _ll: "q", _f: "f", _sz: "N", _vp: "P"}


def _packer(args):
    """Packs a struct's fields, in order, into bytes of its layout: what a call passes, in a
    fraction of the time that filling the ctypes mirror takes."""
    return struct.Struct("@" + "".join(_CODES[t] for _, t in args._fields_) + "0P").pack


class Call:
    """An entry point of the layer operators: ``pack(*fields)`` gives its argument struct as
    bytes, ``fn(bytes, stream)`` is the call, ``size(bytes)`` the workspace that it needs."""

    def __init__(self, lib, name):
        self.name = name
        self.pack = _packer(_LAYER[name])
        self.fn = lib[name]
        self.fn.argtypes, self.fn.restype = [_vp, _vp], ctypes.c_int
        sizes = name + "_workspace_size"
        if sizes in _LAYER_SIZES:
            self._size = lib[sizes]
            self._size.argtypes, self._size.restype = [_vp, _vp], ctypes.c_int

    def size(self, packed):
        n = _sz(0)
        status = self._size(packed, ctypes.byref(n))
        if status:
            check(status, self.name + "_workspace_size")
        return n.value


_calls = {}


def call(name):
    """The Call of a layer operator's entry point."""
    c = _calls.get(name)
    if c is None:
        c = _calls[name] = Call(load(), name)
    return c


# every symbol include/kda.h declares
EXPORTS = ("kda_chunk_fwd_workspace_size", "kda_chunk_fwd", "kda_chunk_fwd_status",
           "kda_chunk_fwd_noalloc", "kda_chunk_fwd_noalloc_status",
           "kda_recurrent_step", "kda_decode_token", "kda_chunk_bwd_workspace_size", "kda_chunk_bwd",
           "kda_status_string", "kda_last_cuda_error", "kda_launch_count", "kda_version", *_LAYER, *_LAYER_SIZES)

_lib = None


def load():
    """Load libkda.so (once) and declare its prototypes."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m kimi_delta_attention_20_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    lib.kda_chunk_fwd_workspace_size.argtypes = [ctypes.POINTER(ChunkArgs),
                                                 ctypes.POINTER(ctypes.c_size_t)]
    lib.kda_chunk_fwd_workspace_size.restype = ctypes.c_int
    lib.kda_chunk_fwd.argtypes = [ctypes.POINTER(ChunkArgs), _vp]
    lib.kda_chunk_fwd.restype = ctypes.c_int
    lib.kda_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(ChunkArgs), _vp]
    lib.kda_chunk_fwd_noalloc.restype = ctypes.c_int
    for name in ("kda_chunk_fwd_status", "kda_chunk_fwd_noalloc_status"):
        getattr(lib, name).argtypes = [ctypes.POINTER(ChunkArgs), _vp]
        getattr(lib, name).restype = ctypes.c_int
    lib.kda_recurrent_step.argtypes = [ctypes.POINTER(StepArgs), _vp]
    lib.kda_recurrent_step.restype = ctypes.c_int
    lib.kda_decode_token.argtypes = [ctypes.POINTER(TokenArgs), _vp]
    lib.kda_decode_token.restype = ctypes.c_int
    lib.kda_chunk_bwd_workspace_size.argtypes = [ctypes.POINTER(BwdArgs), ctypes.POINTER(ctypes.c_size_t)]
    lib.kda_chunk_bwd_workspace_size.restype = ctypes.c_int
    lib.kda_chunk_bwd.argtypes = [ctypes.POINTER(BwdArgs), _vp]
    lib.kda_chunk_bwd.restype = ctypes.c_int
    for name, args in _LAYER.items():
        getattr(lib, name).argtypes = [ctypes.POINTER(args), _vp]
        getattr(lib, name).restype = ctypes.c_int
    for name, args in _LAYER_SIZES.items():
        getattr(lib, name).argtypes = [ctypes.POINTER(args), ctypes.POINTER(_sz)]
        getattr(lib, name).restype = ctypes.c_int
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_last_cuda_error.argtypes = []
    lib.kda_last_cuda_error.restype = ctypes.c_int
    lib.kda_launch_count.argtypes = []
    lib.kda_launch_count.restype = ctypes.c_ulonglong
    lib.kda_version.argtypes = []
    lib.kda_version.restype = ctypes.c_int
    _lib = lib
    return lib


class KDAError(RuntimeError):
    def __init__(self, status: int, what: str):
        lib = load()
        msg = lib.kda_status_string(status).decode()
        if status == KDA_ERR_CUDA:
            msg += f" (cudaError {lib.kda_last_cuda_error()})"
        super().__init__(f"{what}: {msg}")
        self.status = status


def check(status: int, what: str):
    if status != KDA_OK:
        raise KDAError(status, what)
