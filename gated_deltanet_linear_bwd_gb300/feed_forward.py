"""Torch-facing wrappers of the gated feed-forward block, in the manner of layer.py: they check
arguments, allocate outputs and workspace with torch on the tensors' device and pass raw pointers
on the current stream; every computation runs in libgdn.so.
"""
import torch
from torch.autograd.function import once_differentiable

from . import _abi_layer
from .layer import _empty, _empty_like, _first, _grad, _need, _ptr, _with_workspace

_ffn_fwd, _ffn_bwd = _abi_layer.ENTRIES["gdn_ffn_fwd"], _abi_layer.ENTRIES["gdn_ffn_bwd"]

_ACTIVATIONS = {"silu": _abi_layer.GDN_ACT_SILU, "gelu": _abi_layer.GDN_ACT_GELU}


def _block(name, x, w_gate, w_up, w_down, activation):
    """Checks what forward and backward share: (dtype's code, activation's, device index, M, K, F)."""
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r} (silu or gelu)")
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected [..., K]")
    dtype, code, index = _first(name, x)
    if dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {dtype}")
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate has shape {tuple(w_gate.shape)}, expected [F, K]")
    K, F = x.shape[-1], w_gate.shape[0]
    _need("w_gate", w_gate, dtype, (F, K), index)
    _need("w_up", w_up, dtype, (F, K), index)
    _need("w_down", w_down, dtype, (K, F), index)
    return code, act, index, x.numel() // K, K, F


def gated_feed_forward_fwd(x, w_gate, w_up, w_down, activation="silu", save=False):
    """y = (act(x w_gate^T) * (x w_up^T)) w_down^T for x [..., K], w_gate and w_up [F, K] and w_down
    [K, F], all bf16, K and F multiples of 8; activation "silu" or "gelu" (its tanh form).  Returns
    (y, gate, up): with `save` the two projections [..., F] that the backward pass reads, else None."""
    code, act, index, M, K, F = _block("x", x, w_gate, w_up, w_down, activation)
    y = _empty_like(x)
    gate = up = None
    if save:
        gate, up = (_empty((*x.shape[:-1], F), dtype=x.dtype, device=x.device) for _ in range(2))
    _with_workspace(_ffn_fwd, _ffn_fwd.pack(
        x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), M, K, F, code, act, y.data_ptr(),
        _ptr(gate), _ptr(up)), x.device, index)
    return y, gate, up


def gated_feed_forward_bwd(dy, x, w_gate, w_up, w_down, gate, up, activation="silu"):
    """Backward of gated_feed_forward_fwd from its inputs and the projections it saved:
    (dx, dw_gate, dw_up, dw_down), bf16."""
    code, act, index, M, K, F = _block("dy", dy, w_gate, w_up, w_down, activation)
    _need("x", x, dy.dtype, dy.shape, index)
    _need("gate", gate, dy.dtype, (*dy.shape[:-1], F), index)
    _need("up", up, dy.dtype, (*dy.shape[:-1], F), index)
    dx, dwg, dwu, dwd = (_empty_like(t) for t in (x, w_gate, w_up, w_down))
    _with_workspace(_ffn_bwd, _ffn_bwd.pack(
        dy.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), gate.data_ptr(),
        up.data_ptr(), M, K, F, code, act, dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(), dwd.data_ptr()),
        x.device, index)
    return dx, dwg, dwu, dwd


class _GatedFeedForward(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, activation):
        y, gate, up = gated_feed_forward_fwd(x, w_gate, w_up, w_down, activation, save=True)
        ctx.save_for_backward(x, w_gate, w_up, w_down, gate, up)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return *gated_feed_forward_bwd(_grad(dy), *ctx.saved_tensors, activation=ctx.activation), None


def gated_feed_forward(x, w_gate, w_up, w_down, activation="silu"):
    """gated_feed_forward_fwd, differentiable in x and the weights: y.  The projections are kept
    only where a gradient will need them."""
    if not (torch.is_grad_enabled() and any(t.requires_grad for t in (x, w_gate, w_up, w_down))):
        return gated_feed_forward_fwd(x, w_gate, w_up, w_down, activation)[0]
    return _GatedFeedForward.apply(x, w_gate, w_up, w_down, activation)
