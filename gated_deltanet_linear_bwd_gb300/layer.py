"""Torch-facing wrappers of the operators around the gated delta rule: the
residual addition with the RMS norm, microscaled (MX) matrices and their product,
and the per-channel gated linear recurrence.  As in api.py they check arguments,
allocate outputs and workspace with torch on the tensors' device and pass raw
pointers on the current stream; every computation runs in libgdn.so.
"""
import torch
from torch.autograd.function import once_differentiable

from . import _abi_layer
from .api import _DT, _check

# The stream and device of a call, without the Stream and device objects that
# torch.cuda.current_stream() makes (2 us of a decode step's 10)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_empty, _empty_like, _F32, _U8 = torch.empty, torch.empty_like, torch.float32, torch.uint8

_linrec_fwd, _linrec_bwd, _linrec_step, _quantize, _dequantize, _matmul, _linear, _norm_fwd, _norm_bwd = (
    _abi_layer.ENTRIES["gdn_" + name] for name in
    ("linrec_fwd", "linrec_bwd", "linrec_step", "mx_quantize", "mx_dequantize", "mx_matmul",
     "mx_linear", "rms_norm_fwd", "rms_norm_bwd"))


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _grad(t):
    """A gradient as autograd hands it over, contiguous on a 16-byte boundary (a slice of
    another tensor's may be neither); None stays None."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _need(name, t, dtype, shape, index):
    """_check for a tensor that has to be there: contiguous, on device `index`."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        _check(name, t, dtype, shape, torch.device("cuda", index) if index >= 0 else None)
        raise ValueError(f"{name} is not a tensor the library takes")


def _first(name, t):
    """(dtype, its code, device index) of the tensor the others are checked against; its
    device has to be the current one, where the library launches."""
    dtype = t.dtype
    code = _DT.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype} of {name}")
    index = t.get_device()
    if index < 0 or not t.is_contiguous():
        _check(name, t)
    if index != _current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_current_device()}")
    return dtype, code, index


def _with_workspace(entry, packed, dev, index):
    """A call with the workspace it asks for (at most 256 bytes: none)."""
    n = entry.workspace_size(packed)
    if n <= 256:
        entry(packed, 0, 0, _raw_stream(index))
        return
    ws = _empty(n, dtype=_U8, device=dev)
    entry(packed, ws.data_ptr(), n, _raw_stream(index))


# ------------------------------------------------------------------ gated linear recurrence
def _recurrence(name, src, g, initial_state, cu_seqlens, gate_scale):
    """Checks what the forward and backward share: (dtype, its code, device index, B, T, D, N)."""
    if src.dim() != 3:
        raise ValueError(f"expected [B, T, D] tensors, got shape {tuple(src.shape)}")
    dtype, code, index = _first(name, src)
    B, T, D = shape = src.shape
    N = B
    _need("g", g, dtype, shape, index)
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError(f"cu_seqlens has shape {tuple(cu_seqlens.shape)}, expected [N + 1]")
        N = cu_seqlens.numel() - 1
        _need("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), index)
    if initial_state is not None:
        _need("initial_state", initial_state, _F32, (N, D), index)
    if gate_scale is not None:
        _need("gate_scale", gate_scale, torch.float32, (D,), index)
    return dtype, code, index, B, T, D, N


def gated_linear_recurrence_fwd(x, g, initial_state=None, cu_seqlens=None, gate_scale=None,
                                output_final_state=True):
    """h_t = exp(l_t) h_{t-1} + x_t per channel, for x, g [B, T, D] (bf16 or
    fp32): l = g, or -gate_scale softplus(g) with `gate_scale` ([D] fp32).
    States are [N, D] fp32; with `cu_seqlens` ([N + 1] int32) B is 1 and the
    tokens are N packed sequences.  Returns (h, final_state or None)."""
    _, code, index, B, T, D, N = _recurrence("x", x, g, initial_state, cu_seqlens, gate_scale)
    h = _empty_like(x)
    ht = _empty((N, D), dtype=_F32, device=x.device) if output_final_state else None
    _with_workspace(_linrec_fwd, _linrec_fwd.pack(
        x.data_ptr(), g.data_ptr(), _ptr(gate_scale), _ptr(initial_state), _ptr(cu_seqlens), B, T, D,
        N, code, h.data_ptr(), _ptr(ht)), x.device, index)
    return h, ht


def gated_linear_recurrence_bwd(dh, g, h, dht=None, initial_state=None, cu_seqlens=None,
                                gate_scale=None, want_dh0=True):
    """Backward of gated_linear_recurrence_fwd from its output h: returns
    (dx, dg, d(initial_state) or None), and d(gate_scale) as a fourth when
    `gate_scale` is given (dg is then the gradient of the logits)."""
    dtype, code, index, B, T, D, N = _recurrence("dh", dh, g, initial_state, cu_seqlens, gate_scale)
    _need("h", h, dtype, dh.shape, index)
    if dht is not None:
        _need("dht", dht, _F32, (N, D), index)
    dev = dh.device
    dx, dg = _empty_like(dh), _empty_like(dh)
    dh0 = _empty((N, D), dtype=_F32, device=dev) if want_dh0 else None
    ds = None if gate_scale is None else _empty(D, dtype=_F32, device=dev)
    _with_workspace(_linrec_bwd, _linrec_bwd.pack(
        dh.data_ptr(), g.data_ptr(), h.data_ptr(), _ptr(gate_scale), _ptr(initial_state),
        _ptr(cu_seqlens), _ptr(dht), B, T, D, N, code, dx.data_ptr(), dg.data_ptr(), _ptr(dh0),
        _ptr(ds)), dev, index)
    return (dx, dg, dh0) if ds is None else (dx, dg, dh0, ds)


class _GatedLinearRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, initial_state, gate_scale, cu_seqlens):
        h, ht = gated_linear_recurrence_fwd(x, g, initial_state, cu_seqlens, gate_scale)
        ctx.save_for_backward(g, h, initial_state, gate_scale, cu_seqlens)
        return h, ht

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dht):
        g, h, h0, scale, cu = ctx.saved_tensors
        out = gated_linear_recurrence_bwd(_grad(dh), g, h, _grad(dht), h0, cu, scale,
                                          want_dh0=h0 is not None)
        return out[0], out[1], out[2], out[3] if scale is not None else None, None


def gated_linear_recurrence(x, g, initial_state=None, cu_seqlens=None, gate_scale=None,
                            output_final_state=False):
    """gated_linear_recurrence_fwd, differentiable in x, g, initial_state and
    gate_scale: (h, final_state or None)."""
    h, ht = _GatedLinearRecurrence.apply(x, g, initial_state, gate_scale, cu_seqlens)
    return h, (ht if output_final_state else None)


def gated_linear_recurrence_step(x, g, state, gate_scale=None, out_state=None):
    """One token for each of N sequences: x, g [N, D], state [N, D] fp32.
    Returns h [N, D]; the new state goes to `out_state`, or over `state`."""
    if x.dim() != 2:
        raise ValueError(f"expected [N, D] tensors, got shape {tuple(x.shape)}")
    dtype, code, index = _first("x", x)
    N, D = shape = x.shape
    _need("g", g, dtype, shape, index)
    _need("state", state, _F32, shape, index)
    if gate_scale is not None:
        _need("gate_scale", gate_scale, _F32, (D,), index)
    if out_state is None:
        out_state = state
    else:
        _need("out_state", out_state, _F32, shape, index)
    h = _empty_like(x)
    _linrec_step(_linrec_step.pack(
        x.data_ptr(), g.data_ptr(), _ptr(gate_scale), state.data_ptr(), N, D, code,
        h.data_ptr(), out_state.data_ptr()), _raw_stream(index))
    return h


# ------------------------------------------------------------------ microscaled matrices
_FORMATS = {"mxfp8": _abi_layer.GDN_MXFP8, "mxfp4": _abi_layer.GDN_MXFP4}


def _scale_shape(rows, K):
    """Tiles of 128 rows x 4 blocks, indexed [row tile][K tile][row % 32][row / 32][block]."""
    return (-(-rows // 128), -(-K // 128), 32, 4, 4)


class MxTensor:
    """A microscaled matrix [rows, K]: `data` (float8_e4m3fn [rows, K] for "mxfp8",
    uint8 [rows, K / 2] of two e2m1 elements for "mxfp4", the first in the low half)
    and `scales` (uint8 exponents + 127 for each row and 32 columns, in the product's
    order: tiles [row / 128][block / 4][row % 32][row % 128 / 32][block % 4]).  Checked
    when it is made, and not to be changed afterwards."""
    __slots__ = ("_data", "_scales", "_fmt", "_shape", "_index")

    data = property(lambda self: self._data)
    scales = property(lambda self: self._scales)
    fmt = property(lambda self: self._fmt)
    shape = property(lambda self: self._shape)
    device = property(lambda self: self._data.device)

    def __init__(self, data, scales, fmt, shape):
        if fmt not in _FORMATS:
            raise ValueError(f"unknown format {fmt!r} (mxfp8 or mxfp4)")
        rows, K = shape
        if K % 32:
            raise ValueError(f"K = {K}: microscaled matrices take multiples of 32 columns")
        self._data, self._scales, self._fmt, self._shape = data, scales, fmt, (rows, K)
        self._index = index = data.get_device()
        if fmt == "mxfp8":
            _need("data", data, torch.float8_e4m3fn, (rows, K), index)
        else:
            _need("data", data, _U8, (rows, K // 2), index)
        _need("scales", scales, _U8, _scale_shape(rows, K), index)

    @classmethod
    def empty(cls, rows, K, fmt, device):
        if fmt not in _FORMATS:
            raise ValueError(f"unknown format {fmt!r} (mxfp8 or mxfp4)")
        if K % 32:
            raise ValueError(f"K = {K}: microscaled matrices take multiples of 32 columns")
        t = cls.__new__(cls)
        t._data = data = (_empty((rows, K), dtype=torch.float8_e4m3fn, device=device) if fmt == "mxfp8"
                          else _empty((rows, K // 2), dtype=_U8, device=device))
        t._scales = _empty(_scale_shape(rows, K), dtype=_U8, device=device)
        t._fmt, t._shape, t._index = fmt, (rows, K), data.get_device()
        return t


def _mx_index(name, t, index=None):
    """Checks an argument that is to be an MxTensor; its device index (the current
    device's, or `index`)."""
    if type(t) is not MxTensor:
        raise ValueError(f"{name} must be an MxTensor")
    if index is None:
        index = _current_device()
    if t._index != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    return index


def mx_quantize(x, fmt="mxfp4"):
    """x [..., K] (bf16 or fp32) as an MxTensor of [rows, K]: for each row and 32
    columns the least power-of-two scale with which nothing saturates, elements
    rounded to nearest even.  No gradient passes to x."""
    if x.dim() < 1:
        raise ValueError("expected [..., K]")
    _, code, index = _first("x", x)
    K = x.shape[-1]
    rows = x.numel() // K if K else 0
    t = MxTensor.empty(rows, K, fmt, x.device)
    _quantize(_quantize.pack(x.data_ptr(), rows, K, code, _FORMATS[fmt], t._data.data_ptr(),
                             t._scales.data_ptr()), _raw_stream(index))
    return t


def mx_dequantize(t, dtype=torch.float32):
    """The values of an MxTensor, [rows, K] in bf16 or fp32."""
    index = _mx_index("t", t)
    if dtype not in _DT:
        raise ValueError(f"unsupported dtype {dtype}")
    x = torch.empty(t.shape, dtype=dtype, device=t.device)
    _dequantize(_dequantize.pack(t._data.data_ptr(), t._scales.data_ptr(), *t.shape, _DT[dtype],
                                 _FORMATS[t.fmt], x.data_ptr()), _raw_stream(index))
    return x


def mx_from_parts(data, exponents, fmt):
    """An MxTensor from its elements (as MxTensor.data) and row-major scale bytes
    [rows, K / 32], as checkpoints hold them: laid out once, on load."""
    rows, blocks = exponents.shape
    _check("exponents", exponents, torch.uint8, None, data.device)
    R, B = _scale_shape(rows, 32 * blocks)[:2]
    padded = torch.zeros(128 * R, 4 * B, dtype=torch.uint8, device=data.device)
    padded[:rows, :blocks] = exponents
    scales = padded.view(R, 4, 32, B, 4).permute(0, 3, 2, 1, 4).contiguous()
    return MxTensor(data, scales, fmt, (rows, 32 * blocks))


def mx_matmul(a, b, out_dtype=torch.bfloat16):
    """a b^T of MxTensors a [M, K] and b [N, K] of one format: [M, N], summed in fp32.
    No gradients pass through MxTensors."""
    index = _mx_index("a", a)
    _mx_index("b", b, index)
    if a.fmt != b.fmt or a.shape[1] != b.shape[1]:
        raise ValueError(f"a is {a.fmt} {a.shape}, b is {b.fmt} {b.shape}: one format and one K")
    if out_dtype not in _DT:
        raise ValueError(f"unsupported dtype {out_dtype}")
    (M, K), N = a.shape, b.shape[0]
    c = _empty((M, N), dtype=out_dtype, device=a.device)
    _matmul(_matmul.pack(a._data.data_ptr(), a._scales.data_ptr(), b._data.data_ptr(),
                         b._scales.data_ptr(), M, N, K, _FORMATS[a.fmt], _DT[out_dtype],
                         c.data_ptr()), _raw_stream(index))
    return c


class _NoBackward(torch.autograd.Function):
    """mx_linear of a tensor that requires a gradient: the same result, and an error for the
    loss that reaches it."""
    @staticmethod
    def forward(ctx, x, weight, out_dtype):
        return mx_linear(x, weight, out_dtype)

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError("mx_linear has no backward pass: call it under torch.no_grad(), or on x.detach()")


def mx_linear(x, weight, out_dtype=None):
    """x weight^T for x [..., K] (bf16 or fp32, quantised here to the weight's format,
    or an MxTensor of it) and a weight MxTensor [N, K].  Returns [..., N] in x's type
    (bf16 for an MxTensor), or in `out_dtype`.  Forward only: a gradient that reaches it
    raises RuntimeError."""
    if type(x) is MxTensor:
        return mx_matmul(x, weight, out_dtype or torch.bfloat16)
    if x.requires_grad and torch.is_grad_enabled():
        return _NoBackward.apply(x, weight, out_dtype)
    dtype, code, index = _first("x", x)
    _mx_index("weight", weight, index)
    N, K = weight._shape
    shape = x.shape
    if not shape or shape[-1] != K:
        raise ValueError(f"x has shape {tuple(shape)}, the weight {weight.shape}")
    out_code = code
    if out_dtype is None:
        out_dtype = dtype
    else:
        out_code = _DT.get(out_dtype)
        if out_code is None:
            raise ValueError(f"unsupported dtype {out_dtype}")
    dev = x.device
    c = _empty((*shape[:-1], N), dtype=out_dtype, device=dev)
    M = x.numel() // K if K else c.numel() // N if N else 0
    a = _linear.pack(x.data_ptr(), weight._data.data_ptr(), weight._scales.data_ptr(), M, N, K, code,
                     _FORMATS[weight._fmt], out_code, c.data_ptr())
    n = _linear.workspace_size(a)
    ws = _empty(n, dtype=_U8, device=dev)
    _linear(a, ws.data_ptr(), n, _raw_stream(index))
    return c


# ------------------------------------------------------------------ residual addition + RMS norm
def add_rms_norm_fwd(x, weight, residual=None, eps=1e-6, out=None, save_rstd=False):
    """s = x + residual; y = s (mean(s^2) + eps)^-1/2 weight, over the last axis of
    x [..., D] (bf16 or fp32).  Returns (y, s, rstd): y in x's type, or with
    out="mxfp8" an MxTensor of [rows, D]; s in x's type (x itself without a
    residual); rstd [rows] fp32 with save_rstd, else None."""
    shape = x.shape
    if x.dim() < 1 or shape[-1] == 0:
        raise ValueError(f"x has shape {tuple(shape)}, expected [..., D]")
    if out is not None and out != "mxfp8":
        raise ValueError(f"unknown output {out!r} (None or mxfp8)")
    dtype, code, index = _first("x", x)
    D = shape[-1]
    rows = x.numel() // D
    _need("weight", weight, dtype, (D,), index)
    s, sum_ptr = x, 0
    if residual is not None:
        _need("residual", residual, dtype, shape, index)
        s = _empty_like(x)
        sum_ptr = s.data_ptr()
    if out is None:
        y = _empty_like(x)
        y_ptr, scales = y.data_ptr(), 0
    else:
        y = MxTensor.empty(rows, D, out, x.device)
        y_ptr, scales = y._data.data_ptr(), y._scales.data_ptr()
    rstd = _empty(rows, dtype=_F32, device=x.device) if save_rstd else None
    _norm_fwd(_norm_fwd.pack(x.data_ptr(), _ptr(residual), weight.data_ptr(), rows, D, code, eps,
                             out is not None, y_ptr, scales, sum_ptr, _ptr(rstd)), _raw_stream(index))
    return y, s, rstd


def add_rms_norm_bwd(dy, s, weight, rstd, dresidual=None):
    """Backward of add_rms_norm_fwd from its s and rstd: (ds, dweight), ds in dy's type
    (the gradient of x and of the residual), dweight fp32.  `dresidual` is the gradient
    that reaches s past the norm."""
    shape = dy.shape
    if dy.dim() < 1 or shape[-1] == 0:
        raise ValueError(f"dy has shape {tuple(shape)}, expected [..., D]")
    dtype, code, index = _first("dy", dy)
    D = shape[-1]
    rows = dy.numel() // D
    _need("s", s, dtype, shape, index)
    _need("weight", weight, dtype, (D,), index)
    _need("rstd", rstd, _F32, (rows,), index)
    if dresidual is not None:
        _need("dresidual", dresidual, dtype, shape, index)
    dev = dy.device
    ds = _empty_like(dy)
    dw = _empty(D, dtype=_F32, device=dev)
    a = _norm_bwd.pack(dy.data_ptr(), s.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
                       _ptr(dresidual), rows, D, code, ds.data_ptr(), dw.data_ptr())
    n = _norm_bwd.workspace_size(a)
    ws = _empty(n, dtype=_U8, device=dev)
    _norm_bwd(a, ws.data_ptr(), n, _raw_stream(index))
    return ds, dw


class _AddRmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, s, rstd = add_rms_norm_fwd(x, weight, residual, eps, save_rstd=True)
        ctx.save_for_backward(s, weight, rstd)
        ctx.with_residual = residual is not None
        return (y, s) if residual is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds=None):
        s, weight, rstd = ctx.saved_tensors
        d, dw = add_rms_norm_bwd(_grad(dy), s, weight, rstd, _grad(ds))
        return d, dw.to(weight.dtype), d if ctx.with_residual else None, None


def add_rms_norm(x, weight, residual=None, eps=1e-6):
    """add_rms_norm_fwd, differentiable in x, weight and residual: (y, s), or y alone
    without a residual."""
    return _AddRmsNorm.apply(x, weight, residual, eps)
