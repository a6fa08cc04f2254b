"""ctypes binding of the layer operators in libgdn.so (include/gdn_layer.h).
Argument marshalling only; the names mirror the C entry points."""
import ctypes

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


STRUCTS = (gdn_linrec_fwd_args, gdn_linrec_bwd_args, gdn_linrec_step_args)
EXPORTS = ("gdn_linrec_fwd", "gdn_linrec_bwd_workspace_size", "gdn_linrec_bwd",
           "gdn_linrec_step")

_declared = False


def load():
    """libgdn.so with the signatures of gdn_layer.h declared."""
    global _declared
    lib = _abi.load()
    if not _declared:
        p = ctypes.POINTER
        for name, args in (("gdn_linrec_fwd", gdn_linrec_fwd_args),
                           ("gdn_linrec_step", gdn_linrec_step_args)):
            getattr(lib, name).restype = _i32
            getattr(lib, name).argtypes = [p(args), _vp]
        for name, args in (("gdn_linrec_bwd", gdn_linrec_bwd_args),):
            getattr(lib, name).restype = _i32
            getattr(lib, name).argtypes = [p(args), _vp, ctypes.c_size_t, _vp]
            getattr(lib, name + "_workspace_size").restype = ctypes.c_size_t
            getattr(lib, name + "_workspace_size").argtypes = [p(args)]
        _declared = True
    return lib


def call(name: str, args, stream: int) -> None:
    rc = getattr(load(), name)(ctypes.byref(args), stream)
    if rc != GDN_OK:
        raise GdnError(name, rc)


def call_ws(name: str, args, workspace: int, ws_bytes: int, stream: int) -> None:
    rc = getattr(load(), name)(ctypes.byref(args), workspace, ws_bytes, stream)
    if rc != GDN_OK:
        raise GdnError(name, rc)


def workspace_size(name: str, args) -> int:
    n = int(getattr(load(), name + "_workspace_size")(ctypes.byref(args)))
    if n == 0:
        raise GdnError(name + "_workspace_size", GDN_ERR_INVALID_ARG)
    return n
