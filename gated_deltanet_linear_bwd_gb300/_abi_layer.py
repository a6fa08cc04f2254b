"""ctypes binding of the layer operators in libgdn.so (include/gdn_layer.h).
Argument marshalling only; the names mirror the C entry points."""
import ctypes
import struct

from . import _abi
from ._abi import GDN_ERR_INVALID_ARG, GDN_OK, GdnError, _f32, _i32, _vp


class gdn_linrec_fwd_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("g", _vp), ("gate_scale", _vp), ("initial_state", _vp),
                ("cu_seqlens", _vp), ("B", _i32), ("T", _i32), ("D", _i32), ("N", _i32),
                ("dtype", _i32), ("h", _vp), ("final_state", _vp)]


class gdn_linrec_bwd_args(ctypes.Structure):
    _fields_ = [("d_h", _vp), ("g", _vp), ("h", _vp), ("gate_scale", _vp),
                ("initial_state", _vp), ("cu_seqlens", _vp), ("d_final_state", _vp),
                ("B", _i32), ("T", _i32), ("D", _i32), ("N", _i32), ("dtype", _i32),
                ("dx", _vp), ("dg", _vp), ("d_initial_state", _vp), ("d_gate_scale", _vp)]


class gdn_linrec_step_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("g", _vp), ("gate_scale", _vp), ("state", _vp), ("N", _i32),
                ("D", _i32), ("dtype", _i32), ("h", _vp), ("out_state", _vp)]


class gdn_mx_quantize_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("rows", _i32), ("K", _i32), ("dtype", _i32), ("format", _i32),
                ("data", _vp), ("scales", _vp)]


class gdn_mx_dequantize_args(ctypes.Structure):
    _fields_ = [("data", _vp), ("scales", _vp), ("rows", _i32), ("K", _i32), ("dtype", _i32),
                ("format", _i32), ("x", _vp)]


class gdn_mx_matmul_args(ctypes.Structure):
    _fields_ = [("a", _vp), ("a_scales", _vp), ("b", _vp), ("b_scales", _vp), ("M", _i32),
                ("N", _i32), ("K", _i32), ("format", _i32), ("out_dtype", _i32), ("c", _vp)]


class gdn_mx_linear_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("w", _vp), ("w_scales", _vp), ("M", _i32), ("N", _i32), ("K", _i32),
                ("dtype", _i32), ("format", _i32), ("out_dtype", _i32), ("c", _vp)]


class gdn_rms_norm_fwd_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("residual", _vp), ("weight", _vp), ("rows", _i32), ("D", _i32),
                ("dtype", _i32), ("eps", _f32), ("mx", _i32), ("y", _vp), ("scales", _vp),
                ("sum", _vp), ("rstd", _vp)]


class gdn_rms_norm_bwd_args(ctypes.Structure):
    _fields_ = [("dy", _vp), ("sum", _vp), ("weight", _vp), ("rstd", _vp), ("d_sum", _vp),
                ("rows", _i32), ("D", _i32), ("dtype", _i32), ("ds", _vp), ("dweight", _vp)]


GDN_MXFP8, GDN_MXFP4 = 0, 1

_PLAIN = {"gdn_linrec_step": gdn_linrec_step_args,
          "gdn_mx_quantize": gdn_mx_quantize_args, "gdn_mx_dequantize": gdn_mx_dequantize_args,
          "gdn_mx_matmul": gdn_mx_matmul_args, "gdn_rms_norm_fwd": gdn_rms_norm_fwd_args}
_WITH_WORKSPACE = {"gdn_linrec_fwd": gdn_linrec_fwd_args, "gdn_linrec_bwd": gdn_linrec_bwd_args, "gdn_mx_linear": gdn_mx_linear_args,
                   "gdn_rms_norm_bwd": gdn_rms_norm_bwd_args}
STRUCTS = tuple(_PLAIN.values()) + tuple(_WITH_WORKSPACE.values())
EXPORTS = tuple(_PLAIN) + tuple(_WITH_WORKSPACE) + \
    tuple(n + "_workspace_size" for n in _WITH_WORKSPACE) + ("gdn_mx_scale_bytes",)



class Entry:
    """A C entry point.  Its argument struct is packed straight to bytes in the struct's
    own layout (half the time of filling a ctypes.Structure, which a decode step notices):
    `pack` takes the fields in order, addresses as integers (0 for NULL)."""
    _CODES = {_vp: "P", _i32: "i", _f32: "f"}

    def __init__(self, name, fields):
        self.name = name
        self.pack = struct.Struct("@" + "".join(self._CODES[t] for _, t in fields)).pack
        self._call = self._size = None

    def bind(self, lib, with_workspace):
        f = getattr(lib, self.name)
        f.restype = _i32
        f.argtypes = [ctypes.c_char_p] + ([_vp, ctypes.c_size_t] if with_workspace else []) + [_vp]
        self._call = f
        if with_workspace:
            self._size = getattr(lib, self.name + "_workspace_size")
            self._size.restype, self._size.argtypes = ctypes.c_size_t, [ctypes.c_char_p]

    def __call__(self, *args):
        """(packed arguments, [workspace address, bytes,] stream)"""
        rc = self._call(*args)
        if rc != GDN_OK:
            raise GdnError(self.name, rc)

    def workspace_size(self, packed):
        n = self._size(packed)
        if n == 0:
            raise GdnError(self.name + "_workspace_size", GDN_ERR_INVALID_ARG)
        return n


ENTRIES = {name: Entry(name, args._fields_) for name, args in {**_PLAIN, **_WITH_WORKSPACE}.items()}


def load():
    """libgdn.so with the signatures of gdn_layer.h declared."""
    lib = _abi.load()
    if lib.gdn_mx_scale_bytes.argtypes is None:
        for name, entry in ENTRIES.items():
            entry.bind(lib, name in _WITH_WORKSPACE)
        lib.gdn_mx_scale_bytes.restype = ctypes.c_size_t
        lib.gdn_mx_scale_bytes.argtypes = [_i32, _i32]
    return lib
