"""The layer operators' C ABI without a GPU: exports, struct layouts, host-side refusals."""
import ctypes
import os
import re
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_layer.h")


@pytest.fixture(scope="module")
def abi():
    import __graft_entry__
    __graft_entry__.build()
    from gated_deltanet_linear_bwd_gb300 import _abi_layer
    _abi_layer.load()
    return _abi_layer


def test_every_declared_function_is_exported_and_bound(abi):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gdn_[a-z_0-9]+)\s*\(", text))
    assert names == set(abi.EXPORTS)
    for n in names:
        assert hasattr(abi.load(), n), n


def test_struct_layout_matches_header(abi):
    lines = []
    for cls in abi.STRUCTS:
        lines.append(f'  printf("{cls.__name__} sizeof %zu\\n", sizeof({cls.__name__}));')
        lines += [f'  printf("{cls.__name__} {f} %zu\\n", offsetof({cls.__name__}, {f}));' for f, _ in cls._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "gdn_layer.h"\nint main(void) {\n' + "\n".join(lines) + \
        "\n  return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "probe.c"), os.path.join(d, "probe")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-std=c11", "-I", os.path.dirname(HEADER), c, "-o", exe], check=True)
        got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")
    for line in filter(None, got):
        sname, field, val = line.split()
        cls = getattr(abi, sname)
        want = ctypes.sizeof(cls) if field == "sizeof" else getattr(cls, field).offset
        assert want == int(val), line


OK = dict(
    gdn_linrec_fwd=dict(x=4096, g=4096, h=4096, B=2, T=5, D=64),
    gdn_linrec_bwd=dict(d_h=4096, g=4096, h=4096, dx=4096, dg=4096, B=2, T=5, D=64),
    gdn_linrec_step=dict(x=4096, g=4096, state=4096, h=4096, out_state=4096, N=2, D=64),
    gdn_mx_quantize=dict(x=4096, data=4096, scales=4096, rows=3, K=64),
    gdn_mx_dequantize=dict(x=4096, data=4096, scales=4096, rows=3, K=64),
    gdn_mx_matmul=dict(a=4096, a_scales=4096, b=4096, b_scales=4096, c=4096, M=3, N=5, K=64),
    gdn_mx_linear=dict(x=4096, w=4096, w_scales=4096, c=4096, M=3, N=5, K=64),
    gdn_rms_norm_fwd=dict(x=4096, weight=4096, y=4096, rows=3, D=64),
    gdn_rms_norm_bwd=dict(dy=4096, sum=4096, weight=4096, rstd=4096, ds=4096, dweight=4096, rows=3, D=64),
)


def raw(abi, name, **kw):
    a = getattr(abi, name + "_args")()
    for k, v in {**OK[name], **kw}.items():
        setattr(a, k, v)
    return bytes(a)


def call(abi, name, **kw):
    args = raw(abi, name, **kw)
    f = getattr(abi.load(), name)
    return f(args, 4096, 1 << 40, None) if name + "_workspace_size" in abi.EXPORTS else f(args, None)


@pytest.mark.parametrize("name", sorted(OK))
def test_packed_arguments_are_the_structs_bytes(abi, name):
    cls = getattr(abi, name + "_args")
    values = [0.5 if t is ctypes.c_float else 1 + i for i, (_, t) in enumerate(cls._fields_)]
    packed = abi.ENTRIES[name].pack(*values)
    a = cls.from_buffer_copy(packed.ljust(ctypes.sizeof(cls), b"\0"))
    assert [getattr(a, f) for f, _ in cls._fields_] == values


@pytest.mark.parametrize("name, bad, rc, msg", [
    ("gdn_linrec_fwd", dict(B=0), 1, "bad sizes"),
    ("gdn_linrec_fwd", dict(T=-1), 1, "bad sizes"),
    ("gdn_linrec_fwd", dict(dtype=2), 2, "dtype"),
    ("gdn_linrec_fwd", dict(x=None), 1, "required"),
    ("gdn_linrec_fwd", dict(g=4100), 1, "aligned"),
    ("gdn_linrec_fwd", dict(cu_seqlens=4096, N=1), 1, "cu_seqlens"),
    ("gdn_linrec_fwd", dict(cu_seqlens=4096, B=1, N=0), 1, "cu_seqlens"),
    ("gdn_linrec_fwd", dict(B=1 << 16, T=1 << 16), 1, "too large"),
    ("gdn_linrec_bwd", dict(dg=None), 1, "required"),
    ("gdn_linrec_bwd", dict(dx=4104), 1, "aligned"),
    ("gdn_linrec_step", dict(D=0), 1, "bad sizes"),
    ("gdn_linrec_step", dict(out_state=None), 1, "required"),
    ("gdn_mx_quantize", dict(K=48), 2, "multiple of 32"),
    ("gdn_mx_quantize", dict(format=2), 2, "format"),
    ("gdn_mx_quantize", dict(scales=None), 1, "required"),
    ("gdn_mx_dequantize", dict(rows=-1), 1, "bad sizes"),
    ("gdn_mx_matmul", dict(K=40), 2, "multiple of 32"),
    ("gdn_mx_matmul", dict(out_dtype=7), 2, "out_dtype"),
    ("gdn_mx_matmul", dict(b_scales=None), 1, "required"),
    ("gdn_mx_matmul", dict(c=4098), 1, "aligned"),
    ("gdn_mx_matmul", dict(M=-4), 1, "bad sizes"),
    ("gdn_mx_linear", dict(M=-1), 1, "bad sizes"),
    ("gdn_mx_linear", dict(K=40), 2, "multiple of 32"),
    ("gdn_mx_linear", dict(x=None), 1, "required"),
    ("gdn_rms_norm_fwd", dict(D=20000), 2, "16384"),
    ("gdn_rms_norm_fwd", dict(mx=1, scales=4096, D=40), 2, "multiples of 32"),
    ("gdn_rms_norm_fwd", dict(mx=1), 1, "required"),
    ("gdn_rms_norm_fwd", dict(residual=4096), 1, "required"),
    ("gdn_rms_norm_fwd", dict(mx=3), 1, "mx = 3"),
    ("gdn_rms_norm_bwd", dict(rstd=None), 1, "required"),
    ("gdn_rms_norm_bwd", dict(dweight=None), 1, "required"),
])
def test_bad_arguments_are_rejected_on_the_host(abi, name, bad, rc, msg):
    assert call(abi, name, **bad) == rc
    assert msg in abi._abi.gdn_last_error()


def test_null_arguments_and_small_workspaces(abi):
    lib = abi.load()
    for name in OK:
        f = getattr(lib, name)
        rc = f(None, None, 0, None) if name + "_workspace_size" in abi.EXPORTS else f(None, None)
        assert rc == 1
    a = raw(abi, "gdn_rms_norm_bwd")
    need = abi.ENTRIES["gdn_rms_norm_bwd"].workspace_size(a)
    assert need >= 256
    assert lib.gdn_rms_norm_bwd(a, 4096, need - 1, None) == 3
    for name, kw in (("gdn_linrec_bwd", dict(gate_scale=4096, d_gate_scale=4096)),
                     ("gdn_linrec_fwd", dict(B=1, T=60000)), ("gdn_mx_linear", {})):
        a = raw(abi, name, **kw)
        need = abi.ENTRIES[name].workspace_size(a)
        assert need > 256 or name == "gdn_mx_linear"
        f = getattr(lib, name)
        assert f(a, None, 0, None) == 3 and f(a, 4096, need - 1, None) == 3 and f(a, 4100, need, None) == 3


def test_empty_problems_are_host_side_no_ops(abi):
    assert call(abi, "gdn_linrec_step", N=0) == 0
    assert call(abi, "gdn_mx_quantize", rows=0) == 0
    assert call(abi, "gdn_mx_matmul", M=0) == 0
    assert call(abi, "gdn_rms_norm_fwd", rows=0) == 0


def test_scale_bytes(abi):
    f = abi.load().gdn_mx_scale_bytes
    assert [f(1, 32), f(128, 128), f(129, 160), f(0, 64), f(5, 0)] == [512, 512, 2048, 0, 0]
