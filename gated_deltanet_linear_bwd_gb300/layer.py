"""Torch-facing wrappers of the operators around the gated delta rule: the
residual addition with the RMS norm, microscaled (MX) matrices and their product,
and the per-channel gated linear recurrence.  As in api.py they check arguments,
allocate outputs and workspace with torch on the tensors' device and pass raw
pointers on the current stream; every computation runs in libgdn.so.
"""
import torch

from . import _abi_layer
from .api import _DT, _check, _ptr

# The stream and device of a call, without the Stream and device objects that
# torch.cuda.current_stream() makes (2 us of a decode step's 10)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _need(name, t, dtype, shape, index):
    """_check for a tensor that has to be there: contiguous, on device `index`."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        _check(name, t, dtype, shape, torch.device("cuda", index) if index >= 0 else None)
        raise ValueError(f"{name} is not a tensor the library takes")


def _first(name, t):
    """(dtype, device index) of the tensor the others are checked against; its device
    has to be the current one, where the library launches."""
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype} of {name}")
    index = t.get_device()
    if index < 0 or not t.is_contiguous():
        _check(name, t)
    if index != _current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_current_device()}")
    return t.dtype, index


def _with_workspace(name, args, dev, index):
    """A call with the workspace it asks for (at most 256 bytes: none)."""
    n = _abi_layer.workspace_size(name, args)
    if n <= 256:
        _abi_layer.call_ws(name, args, 0, 0, _raw_stream(index))
        return
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _abi_layer.call_ws(name, args, ws.data_ptr(), n, _raw_stream(index))


# ------------------------------------------------------------------ gated linear recurrence
def _recurrence(name, src, g, initial_state, cu_seqlens, gate_scale):
    """Checks what the forward and backward share: (dtype, device index, B, T, D, N)."""
    if src.dim() != 3:
        raise ValueError(f"expected [B, T, D] tensors, got shape {tuple(src.shape)}")
    dtype, index = _first(name, src)
    B, T, D = shape = src.shape
    N = B
    _need("g", g, dtype, shape, index)
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError(f"cu_seqlens has shape {tuple(cu_seqlens.shape)}, expected [N + 1]")
        N = cu_seqlens.numel() - 1
        _need("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), index)
    if initial_state is not None:
        _need("initial_state", initial_state, torch.float32, (N, D), index)
    if gate_scale is not None:
        _need("gate_scale", gate_scale, torch.float32, (D,), index)
    return dtype, index, B, T, D, N


def gated_linear_recurrence_fwd(x, g, initial_state=None, cu_seqlens=None, gate_scale=None,
                                output_final_state=True):
    """h_t = exp(l_t) h_{t-1} + x_t per channel, for x, g [B, T, D] (bf16 or
    fp32): l = g, or -gate_scale softplus(g) with `gate_scale` ([D] fp32).
    States are [N, D] fp32; with `cu_seqlens` ([N + 1] int32) B is 1 and the
    tokens are N packed sequences.  Returns (h, final_state or None)."""
    dtype, index, B, T, D, N = _recurrence("x", x, g, initial_state, cu_seqlens, gate_scale)
    h = torch.empty_like(x)
    ht = torch.empty((N, D), dtype=torch.float32, device=x.device) if output_final_state else None
    _with_workspace("gdn_linrec_fwd", _abi_layer.gdn_linrec_fwd_args(
        x.data_ptr(), g.data_ptr(), _ptr(gate_scale), _ptr(initial_state), _ptr(cu_seqlens), B, T, D,
        N, _DT[dtype], h.data_ptr(), _ptr(ht)), x.device, index)
    return h, ht


def gated_linear_recurrence_bwd(dh, g, h, dht=None, initial_state=None, cu_seqlens=None,
                                gate_scale=None, want_dh0=True):
    """Backward of gated_linear_recurrence_fwd from its output h: returns
    (dx, dg, d(initial_state) or None), and d(gate_scale) as a fourth when
    `gate_scale` is given (dg is then the gradient of the logits)."""
    dtype, index, B, T, D, N = _recurrence("dh", dh, g, initial_state, cu_seqlens, gate_scale)
    _need("h", h, dtype, dh.shape, index)
    if dht is not None:
        _need("dht", dht, torch.float32, (N, D), index)
    dev = dh.device
    dx, dg = torch.empty_like(dh), torch.empty_like(dh)
    dh0 = torch.empty((N, D), dtype=torch.float32, device=dev) if want_dh0 else None
    ds = None if gate_scale is None else torch.empty(D, dtype=torch.float32, device=dev)
    a = _abi_layer.gdn_linrec_bwd_args(
        dh.data_ptr(), g.data_ptr(), h.data_ptr(), _ptr(gate_scale), _ptr(initial_state),
        _ptr(cu_seqlens), _ptr(dht), B, T, D, N, _DT[dtype], dx.data_ptr(), dg.data_ptr(), _ptr(dh0),
        _ptr(ds))
    _with_workspace("gdn_linrec_bwd", a, dev, index)
    return (dx, dg, dh0) if ds is None else (dx, dg, dh0, ds)


class _GatedLinearRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, initial_state, gate_scale, cu_seqlens):
        h, ht = gated_linear_recurrence_fwd(x, g, initial_state, cu_seqlens, gate_scale)
        ctx.save_for_backward(g, h, initial_state, gate_scale, cu_seqlens)
        return h, ht

    @staticmethod
    def backward(ctx, dh, dht):
        g, h, h0, scale, cu = ctx.saved_tensors
        out = gated_linear_recurrence_bwd(dh.contiguous(), g, h, dht.contiguous(), h0, cu, scale,
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
    dtype, index = _first("x", x)
    N, D = shape = x.shape
    _need("g", g, dtype, shape, index)
    _need("state", state, torch.float32, shape, index)
    if gate_scale is not None:
        _need("gate_scale", gate_scale, torch.float32, (D,), index)
    if out_state is None:
        out_state = state
    else:
        _need("out_state", out_state, torch.float32, shape, index)
    h = torch.empty_like(x)
    _abi_layer.call("gdn_linrec_step", _abi_layer.gdn_linrec_step_args(
        x.data_ptr(), g.data_ptr(), _ptr(gate_scale), state.data_ptr(), N, D, _DT[dtype],
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
    order: tiles [row / 128][block / 4][row % 32][row % 128 / 32][block % 4])."""
    __slots__ = ("data", "scales", "fmt", "shape")

    def __init__(self, data, scales, fmt, shape):
        self.data, self.scales, self.fmt, self.shape = data, scales, fmt, shape

    @classmethod
    def empty(cls, rows, K, fmt, device):
        if fmt not in _FORMATS:
            raise ValueError(f"unknown format {fmt!r} (mxfp8 or mxfp4)")
        if K % 32:
            raise ValueError(f"K = {K}: microscaled matrices take multiples of 32 columns")
        data = (torch.empty((rows, K), dtype=torch.float8_e4m3fn, device=device) if fmt == "mxfp8"
                else torch.empty((rows, K // 2), dtype=torch.uint8, device=device))
        return cls(data, torch.empty(_scale_shape(rows, K), dtype=torch.uint8, device=device), fmt,
                   (rows, K))

    @property
    def device(self):
        return self.data.device


def _mx_index(name, t, index=None):
    """Checks an MxTensor; its device index (the current device's, or `index`)."""
    if not isinstance(t, MxTensor):
        raise ValueError(f"{name} must be an MxTensor")
    rows, K = t.shape
    if index is None:
        index = t.data.get_device()
        if index >= 0 and index != _current_device():
            raise ValueError(f"{name} is on cuda:{index}, the current device is cuda:{_current_device()}")
    if t.fmt == "mxfp8":
        _need(name + ".data", t.data, torch.float8_e4m3fn, (rows, K), index)
    else:
        _need(name + ".data", t.data, torch.uint8, (rows, K // 2), index)
    _need(name + ".scales", t.scales, torch.uint8, _scale_shape(rows, K), index)
    return index


def mx_quantize(x, fmt="mxfp4"):
    """x [..., K] (bf16 or fp32) as an MxTensor of [rows, K]: for each row and 32
    columns the least power-of-two scale with which nothing saturates, elements
    rounded to nearest even."""
    if x.dim() < 1:
        raise ValueError("expected [..., K]")
    dtype, index = _first("x", x)
    K = x.shape[-1]
    rows = x.numel() // K if K else 0
    t = MxTensor.empty(rows, K, fmt, x.device)
    _abi_layer.call("gdn_mx_quantize", _abi_layer.gdn_mx_quantize_args(
        x.data_ptr(), rows, K, _DT[dtype], _FORMATS[fmt], t.data.data_ptr(), t.scales.data_ptr()),
        _raw_stream(index))
    return t


def mx_dequantize(t, dtype=torch.float32):
    """The values of an MxTensor, [rows, K] in bf16 or fp32."""
    index = _mx_index("t", t)
    if dtype not in _DT:
        raise ValueError(f"unsupported dtype {dtype}")
    x = torch.empty(t.shape, dtype=dtype, device=t.device)
    _abi_layer.call("gdn_mx_dequantize", _abi_layer.gdn_mx_dequantize_args(
        t.data.data_ptr(), t.scales.data_ptr(), *t.shape, _DT[dtype], _FORMATS[t.fmt], x.data_ptr()),
        _raw_stream(index))
    return x


def mx_from_parts(data, exponents, fmt):
    """An MxTensor from its elements (as MxTensor.data) and row-major scale bytes
    [rows, K / 32], as checkpoints hold them: laid out once, on load."""
    rows, blocks = exponents.shape
    t = MxTensor.empty(rows, 32 * blocks, fmt, data.device)
    _check("exponents", exponents, torch.uint8, None, data.device)
    _check("data", data, t.data.dtype, tuple(t.data.shape))
    R, B = t.scales.shape[:2]
    padded = torch.zeros(128 * R, 4 * B, dtype=torch.uint8, device=data.device)
    padded[:rows, :blocks] = exponents
    t.scales.copy_(padded.view(R, 4, 32, B, 4).permute(0, 3, 2, 1, 4))
    t.data = data
    return t


def mx_matmul(a, b, out_dtype=torch.bfloat16):
    """a b^T of MxTensors a [M, K] and b [N, K] of one format: [M, N], summed in fp32."""
    index = _mx_index("a", a)
    _mx_index("b", b, index)
    if a.fmt != b.fmt or a.shape[1] != b.shape[1]:
        raise ValueError(f"a is {a.fmt} {a.shape}, b is {b.fmt} {b.shape}: one format and one K")
    if out_dtype not in _DT:
        raise ValueError(f"unsupported dtype {out_dtype}")
    (M, K), N = a.shape, b.shape[0]
    c = torch.empty((M, N), dtype=out_dtype, device=a.device)
    _abi_layer.call("gdn_mx_matmul", _abi_layer.gdn_mx_matmul_args(
        a.data.data_ptr(), a.scales.data_ptr(), b.data.data_ptr(), b.scales.data_ptr(), M, N, K,
        _FORMATS[a.fmt], _DT[out_dtype], c.data_ptr()), _raw_stream(index))
    return c


def mx_linear(x, weight, out_dtype=None):
    """x weight^T for x [..., K] (bf16 or fp32, quantised here to the weight's format,
    or an MxTensor of it) and a weight MxTensor [N, K].  Returns [..., N] in x's type
    (bf16 for an MxTensor), or in `out_dtype`."""
    if isinstance(x, MxTensor):
        return mx_matmul(x, weight, out_dtype or torch.bfloat16)
    dtype, index = _first("x", x)
    _mx_index("weight", weight, index)
    N, K = weight.shape
    if x.dim() < 1 or x.shape[-1] != K:
        raise ValueError(f"x has shape {tuple(x.shape)}, the weight {weight.shape}")
    out_dtype = out_dtype or dtype
    if out_dtype not in _DT:
        raise ValueError(f"unsupported dtype {out_dtype}")
    shape, dev = (*x.shape[:-1], N), x.device
    c = torch.empty(shape, dtype=out_dtype, device=dev)
    M = c.numel() // N if N else 0
    a = _abi_layer.gdn_mx_linear_args(x.data_ptr(), weight.data.data_ptr(), weight.scales.data_ptr(),
                                      M, N, K, _DT[dtype], _FORMATS[weight.fmt], _DT[out_dtype],
                                      c.data_ptr())
    n = _abi_layer.workspace_size("gdn_mx_linear", a)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _abi_layer.call_ws("gdn_mx_linear", a, ws.data_ptr(), n, _raw_stream(index))
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
    dtype, index = _first("x", x)
    D = shape[-1]
    rows = x.numel() // D
    _need("weight", weight, dtype, (D,), index)
    s, sum_ptr = x, None
    if residual is not None:
        _need("residual", residual, dtype, shape, index)
        s = torch.empty_like(x)
        sum_ptr = s.data_ptr()
    if out is None:
        y = torch.empty_like(x)
        y_ptr, scales = y.data_ptr(), None
    else:
        y = MxTensor.empty(rows, D, out, x.device)
        y_ptr, scales = y.data.data_ptr(), y.scales.data_ptr()
    rstd = torch.empty(rows, dtype=torch.float32, device=x.device) if save_rstd else None
    _abi_layer.call("gdn_rms_norm_fwd", _abi_layer.gdn_rms_norm_fwd_args(
        x.data_ptr(), _ptr(residual), weight.data_ptr(), rows, D, _DT[dtype], eps, out is not None,
        y_ptr, scales, sum_ptr, _ptr(rstd)), _raw_stream(index))
    return y, s, rstd


def add_rms_norm_bwd(dy, s, weight, rstd, dresidual=None):
    """Backward of add_rms_norm_fwd from its s and rstd: (ds, dweight), ds in dy's type
    (the gradient of x and of the residual), dweight fp32.  `dresidual` is the gradient
    that reaches s past the norm."""
    shape = dy.shape
    if dy.dim() < 1 or shape[-1] == 0:
        raise ValueError(f"dy has shape {tuple(shape)}, expected [..., D]")
    dtype, index = _first("dy", dy)
    D = shape[-1]
    rows = dy.numel() // D
    _need("s", s, dtype, shape, index)
    _need("weight", weight, dtype, (D,), index)
    _need("rstd", rstd, torch.float32, (rows,), index)
    if dresidual is not None:
        _need("dresidual", dresidual, dtype, shape, index)
    dev = dy.device
    ds = torch.empty_like(dy)
    dw = torch.empty(D, dtype=torch.float32, device=dev)
    a = _abi_layer.gdn_rms_norm_bwd_args(dy.data_ptr(), s.data_ptr(), weight.data_ptr(),
                                         rstd.data_ptr(), _ptr(dresidual), rows, D, _DT[dtype],
                                         ds.data_ptr(), dw.data_ptr())
    n = _abi_layer.workspace_size("gdn_rms_norm_bwd", a)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _abi_layer.call_ws("gdn_rms_norm_bwd", a, ws.data_ptr(), n, _raw_stream(index))
    return ds, dw


class _AddRmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, s, rstd = add_rms_norm_fwd(x, weight, residual, eps, save_rstd=True)
        ctx.save_for_backward(s, weight, rstd)
        ctx.with_residual = residual is not None
        return (y, s) if residual is not None else y

    @staticmethod
    def backward(ctx, dy, ds=None):
        s, weight, rstd = ctx.saved_tensors
        d, dw = add_rms_norm_bwd(dy.contiguous(), s, weight, rstd,
                                 None if ds is None else ds.contiguous())
        return d, dw.to(weight.dtype), d if ctx.with_residual else None, None


def add_rms_norm(x, weight, residual=None, eps=1e-6):
    """add_rms_norm_fwd, differentiable in x, weight and residual: (y, s), or y alone
    without a residual."""
    return _AddRmsNorm.apply(x, weight, residual, eps)
