"""Torch-facing wrappers of the short causal convolution and the selective state space scan, in the
manner of layer.py: they check
arguments, allocate outputs and workspace with torch on the tensors' device and pass raw pointers
on the current stream; every computation runs in libgdn.so.
"""
import torch
from torch.autograd.function import once_differentiable

from . import _abi_layer
from .layer import _F32, _empty, _empty_like, _first, _grad, _need, _ptr, _raw_stream, _with_workspace

_conv_fwd, _conv_bwd, _conv_step = (_abi_layer.ENTRIES["gdn_" + name] for name in ("conv_fwd", "conv_bwd", "conv_step"))
_ssm_fwd, _ssm_bwd, _ssm_step = (_abi_layer.ENTRIES["gdn_" + name] for name in ("ssm_fwd", "ssm_bwd", "ssm_step"))

_ACTIVATIONS = {None: _abi_layer.GDN_ACT_NONE, "silu": _abi_layer.GDN_ACT_SILU}


def _activation(name):
    code = _ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"unknown activation {name!r} (None or silu)")
    return code


def _sequences(name, src, cu_seqlens):
    """(dtype, its code, device index, B, T, D, N) of a [B, T, D] tensor, or of N packed sequences."""
    if src.dim() != 3:
        raise ValueError(f"expected [B, T, D] tensors, got shape {tuple(src.shape)}")
    dtype, code, index = _first(name, src)
    B, T, D = src.shape
    N = B
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError(f"cu_seqlens has shape {tuple(cu_seqlens.shape)}, expected [N + 1]")
        N = cu_seqlens.numel() - 1
        _need("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), index)
    return dtype, code, index, B, T, D, N


# ------------------------------------------------------------------ short causal convolution
def _taps(weight, bias, dtype, D, index):
    """The number of taps of weight [D, W], bias checked with it."""
    if weight.dim() != 2:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected [D, W]")
    W = weight.shape[1]
    _need("weight", weight, dtype, (D, W), index)
    if bias is not None:
        _need("bias", bias, dtype, (D,), index)
    if not 2 <= W <= 4:
        raise ValueError(f"weight has {W} taps (2 to 4)")
    return W


def causal_convolution_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation="silu",
                           output_final_state=True):
    """y_t = act(bias + sum_k weight[:, k] x_{t - W + 1 + k}) per channel, for x [B, T, D] (bf16 or
    fp32) and weight [D, W], W = 2 to 4; activation "silu" or None.  States are the W - 1 inputs
    before a sequence, [N, W - 1, D] in x's type, oldest first (zeros without initial_state); with
    `cu_seqlens` ([N + 1] int32) B is 1 and the tokens are N packed sequences.  Returns
    (y, final_state or None)."""
    act = _activation(activation)
    dtype, code, index, B, T, D, N = _sequences("x", x, cu_seqlens)
    W = _taps(weight, bias, dtype, D, index)
    if initial_state is not None:
        _need("initial_state", initial_state, dtype, (N, W - 1, D), index)
    y = _empty_like(x)
    ht = _empty((N, W - 1, D), dtype=dtype, device=x.device) if output_final_state else None
    _conv_fwd(_conv_fwd.pack(x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(initial_state), _ptr(cu_seqlens),
                             B, T, D, N, W, code, act, y.data_ptr(), _ptr(ht)), _raw_stream(index))
    return y, ht


def causal_convolution_bwd(dy, x, weight, bias=None, dht=None, initial_state=None, cu_seqlens=None,
                           activation="silu", want_dh0=True):
    """Backward of causal_convolution_fwd from its inputs: (dx, dweight, dbias or None,
    d(initial_state) or None); dx and d(initial_state) in x's type, dweight [D, W] and dbias [D]
    (with a bias) fp32.  `dht` is the gradient of the final state."""
    act = _activation(activation)
    dtype, code, index, B, T, D, N = _sequences("dy", dy, cu_seqlens)
    W = _taps(weight, bias, dtype, D, index)
    _need("x", x, dtype, dy.shape, index)
    if dht is not None:
        _need("dht", dht, dtype, (N, W - 1, D), index)
    if initial_state is not None:
        _need("initial_state", initial_state, dtype, (N, W - 1, D), index)
    dev = dy.device
    dx = _empty_like(dy)
    dw = _empty((D, W), dtype=_F32, device=dev)
    db = None if bias is None else _empty(D, dtype=_F32, device=dev)
    dh0 = _empty((N, W - 1, D), dtype=dtype, device=dev) if want_dh0 else None
    _with_workspace(_conv_bwd, _conv_bwd.pack(
        dy.data_ptr(), x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(initial_state), _ptr(cu_seqlens), _ptr(dht),
        B, T, D, N, W, code, act, dx.data_ptr(), dw.data_ptr(), _ptr(db), _ptr(dh0)), dev, index)
    return dx, dw, db, dh0


class _CausalConvolution(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, cu_seqlens, activation):
        y, ht = causal_convolution_fwd(x, weight, bias, initial_state, cu_seqlens, activation)
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.activation = activation
        return y, ht

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dht):
        x, weight, bias, h0, cu = ctx.saved_tensors
        dx, dw, db, dh0 = causal_convolution_bwd(_grad(dy), x, weight, bias, _grad(dht), h0, cu, ctx.activation,
                                                 want_dh0=h0 is not None)
        return dx, dw.to(weight.dtype), None if db is None else db.to(bias.dtype), dh0, None, None


def causal_convolution(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation="silu",
                       output_final_state=False):
    """causal_convolution_fwd, differentiable in x, weight, bias and initial_state:
    (y, final_state or None)."""
    y, ht = _CausalConvolution.apply(x, weight, bias, initial_state, cu_seqlens, activation)
    return y, (ht if output_final_state else None)


def causal_convolution_step(x, weight, state, bias=None, activation="silu", out_state=None):
    """One token for each of N sequences: x [N, D], state [N, W - 1, D] in x's type.  Returns
    y [N, D]; the new state goes to `out_state`, or over `state`."""
    act = _activation(activation)
    if x.dim() != 2:
        raise ValueError(f"expected [N, D] tensors, got shape {tuple(x.shape)}")
    dtype, code, index = _first("x", x)
    N, D = x.shape
    W = _taps(weight, bias, dtype, D, index)
    _need("state", state, dtype, (N, W - 1, D), index)
    if out_state is None:
        out_state = state
    else:
        _need("out_state", out_state, dtype, (N, W - 1, D), index)
    y = _empty_like(x)
    _conv_step(_conv_step.pack(x.data_ptr(), weight.data_ptr(), _ptr(bias), state.data_ptr(), N, D, W, code, act,
                               y.data_ptr(), out_state.data_ptr()), _raw_stream(index))
    return y


# ------------------------------------------------------------------ selective state space scan
def _scan_inputs(dtype, lead, D, index, dt, a, b, c, skip, z, dt_bias):
    """Checks what the scan and the step share; the number of states."""
    if a.dim() != 2:
        raise ValueError(f"a has shape {tuple(a.shape)}, expected [D, S]")
    S = a.shape[1]
    if not 1 <= S <= 64:
        raise ValueError(f"a has {S} states (1 to 64)")
    _need("dt", dt, dtype, (*lead, D), index)
    _need("a", a, _F32, (D, S), index)
    _need("b", b, dtype, (*lead, S), index)
    _need("c", c, dtype, (*lead, S), index)
    if skip is not None:
        _need("skip", skip, _F32, (D,), index)
    if z is not None:
        _need("z", z, dtype, (*lead, D), index)
    if dt_bias is not None:
        _need("dt_bias", dt_bias, _F32, (D,), index)
    return S


def state_space_scan_fwd(x, dt, a, b, c, skip=None, z=None, dt_bias=None, initial_state=None, cu_seqlens=None,
                         output_final_state=True):
    """h_t = exp(delta_t a) h_{t-1} + delta_t x_t b_t and y_t = (<c_t, h_t> + skip x_t) silu(z_t), for
    each channel of x, dt, z [B, T, D] and its S states (1 to 64); b, c [B, T, S] in x's type (bf16 or
    fp32), a [D, S] and skip [D] fp32.  delta = dt, or softplus(dt + dt_bias) with `dt_bias` ([D]
    fp32).  States are [N, D, S] fp32; with `cu_seqlens` ([N + 1] int32) B is 1 and the tokens are N
    packed sequences.  Returns (y, final_state or None)."""
    dtype, code, index, B, T, D, N = _sequences("x", x, cu_seqlens)
    S = _scan_inputs(dtype, (B, T), D, index, dt, a, b, c, skip, z, dt_bias)
    if initial_state is not None:
        _need("initial_state", initial_state, _F32, (N, D, S), index)
    y = _empty_like(x)
    ht = _empty((N, D, S), dtype=_F32, device=x.device) if output_final_state else None
    _with_workspace(_ssm_fwd, _ssm_fwd.pack(
        x.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(), _ptr(skip), _ptr(z), _ptr(dt_bias),
        _ptr(initial_state), _ptr(cu_seqlens), B, T, D, S, N, code, y.data_ptr(), _ptr(ht)), x.device, index)
    return y, ht


def state_space_scan_bwd(dy, x, dt, a, b, c, skip=None, z=None, dt_bias=None, dht=None, initial_state=None,
                         cu_seqlens=None, want_dh0=True):
    """Backward of state_space_scan_fwd from its inputs: (dx, ddt, da, db, dc, dskip, dz, ddt_bias,
    d(initial_state)), None for what was not given (or not wanted); da, dskip, ddt_bias and
    d(initial_state) fp32, the others in x's type.  `dht` is the gradient of the final state."""
    dtype, code, index, B, T, D, N = _sequences("dy", dy, cu_seqlens)
    _need("x", x, dtype, dy.shape, index)
    S = _scan_inputs(dtype, (B, T), D, index, dt, a, b, c, skip, z, dt_bias)
    if initial_state is not None:
        _need("initial_state", initial_state, _F32, (N, D, S), index)
    if dht is not None:
        _need("dht", dht, _F32, (N, D, S), index)
    dx, ddt, da, db, dc = (_empty_like(t) for t in (x, dt, a, b, c))
    dskip, dz, dbias = (None if t is None else _empty_like(t) for t in (skip, z, dt_bias))
    dh0 = _empty((N, D, S), dtype=_F32, device=x.device) if want_dh0 else None
    _with_workspace(_ssm_bwd, _ssm_bwd.pack(
        dy.data_ptr(), x.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(), _ptr(skip), _ptr(z),
        _ptr(dt_bias), _ptr(initial_state), _ptr(cu_seqlens), _ptr(dht), B, T, D, S, N, code, dx.data_ptr(),
        ddt.data_ptr(), da.data_ptr(), db.data_ptr(), dc.data_ptr(), _ptr(dskip), _ptr(dz), _ptr(dbias), _ptr(dh0)),
        x.device, index)
    return dx, ddt, da, db, dc, dskip, dz, dbias, dh0


class _StateSpaceScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, a, b, c, skip, z, dt_bias, initial_state, cu_seqlens):
        y, ht = state_space_scan_fwd(x, dt, a, b, c, skip, z, dt_bias, initial_state, cu_seqlens)
        ctx.save_for_backward(x, dt, a, b, c, skip, z, dt_bias, initial_state, cu_seqlens)
        return y, ht

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dht):
        *inputs, h0, cu = ctx.saved_tensors
        return *state_space_scan_bwd(_grad(dy), *inputs, dht=_grad(dht), initial_state=h0, cu_seqlens=cu,
                                     want_dh0=h0 is not None), None


def state_space_scan(x, dt, a, b, c, skip=None, z=None, dt_bias=None, initial_state=None, cu_seqlens=None,
                     output_final_state=False):
    """state_space_scan_fwd, differentiable in all but cu_seqlens: (y, final_state or None)."""
    y, ht = _StateSpaceScan.apply(x, dt, a, b, c, skip, z, dt_bias, initial_state, cu_seqlens)
    return y, (ht if output_final_state else None)


def state_space_step(x, dt, a, b, c, state, skip=None, z=None, dt_bias=None, out_state=None):
    """One token for each of N sequences: x, dt, z [N, D], b, c [N, S], state [N, D, S] fp32.
    Returns y [N, D]; the new state goes to `out_state`, or over `state`."""
    if x.dim() != 2:
        raise ValueError(f"expected [N, D] tensors, got shape {tuple(x.shape)}")
    dtype, code, index = _first("x", x)
    N, D = x.shape
    S = _scan_inputs(dtype, (N,), D, index, dt, a, b, c, skip, z, dt_bias)
    _need("state", state, _F32, (N, D, S), index)
    if out_state is None:
        out_state = state
    else:
        _need("out_state", out_state, _F32, (N, D, S), index)
    y = _empty_like(x)
    _ssm_step(_ssm_step.pack(
        x.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(), _ptr(skip), _ptr(z), _ptr(dt_bias),
        state.data_ptr(), N, D, S, code, y.data_ptr(), out_state.data_ptr()), _raw_stream(index))
    return y
