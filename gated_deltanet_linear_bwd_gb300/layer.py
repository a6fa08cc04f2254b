"""Torch-facing wrappers of the operators around the gated delta rule: the
per-channel gated linear recurrence.  As in api.py they check arguments,
allocate outputs and workspace with torch on the tensors' device and pass raw
pointers on the current stream; every computation runs in libgdn.so.
"""
import torch

from . import _abi_layer
from .api import _DT, _check, _ptr


def _stream(dev):
    """The current stream of `dev`, which has to be the current device: the
    library launches there."""
    if torch.cuda.current_device() != dev.index:
        raise ValueError(f"the tensors are on {dev}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return torch.cuda.current_stream(dev).cuda_stream


def _dtype(name, t):
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype} of {name}")
    return _DT[t.dtype]


# ------------------------------------------------------------------ gated linear recurrence
def _recurrence(args, src, g, initial_state, cu_seqlens, gate_scale):
    if src.dim() != 3:
        raise ValueError(f"expected [B, T, D] tensors, got shape {tuple(src.shape)}")
    args.dtype = _dtype("the input", src)
    B, T, D = src.shape
    dev = src.device
    if cu_seqlens is not None and (cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2):
        raise ValueError(f"cu_seqlens has shape {tuple(cu_seqlens.shape)}, expected [N + 1]")
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    _check("g", g, src.dtype, (B, T, D), dev)
    _check("initial_state", initial_state, torch.float32, (N, D), dev)
    _check("cu_seqlens", cu_seqlens, torch.int32, None, dev)
    _check("gate_scale", gate_scale, torch.float32, (D,), dev)
    args.g, args.gate_scale = g.data_ptr(), _ptr(gate_scale)
    args.initial_state, args.cu_seqlens = _ptr(initial_state), _ptr(cu_seqlens)
    args.B, args.T, args.D, args.N = B, T, D, N
    return B, T, D, N, dev


def gated_linear_recurrence_fwd(x, g, initial_state=None, cu_seqlens=None, gate_scale=None,
                                output_final_state=True):
    """h_t = exp(l_t) h_{t-1} + x_t per channel, for x, g [B, T, D] (bf16 or
    fp32): l = g, or -gate_scale softplus(g) with `gate_scale` ([D] fp32).
    States are [N, D] fp32; with `cu_seqlens` ([N + 1] int32) B is 1 and the
    tokens are N packed sequences.  Returns (h, final_state or None)."""
    a = _abi_layer.gdn_linrec_fwd_args()
    _check("x", x)
    B, T, D, N, dev = _recurrence(a, x, g, initial_state, cu_seqlens, gate_scale)
    h = torch.empty_like(x)
    ht = torch.empty(N, D, dtype=torch.float32, device=dev) if output_final_state else None
    a.x, a.h, a.final_state = x.data_ptr(), h.data_ptr(), _ptr(ht)
    _abi_layer.call("gdn_linrec_fwd", a, _stream(dev))
    return h, ht


def gated_linear_recurrence_bwd(dh, g, h, dht=None, initial_state=None, cu_seqlens=None,
                                gate_scale=None, want_dh0=True):
    """Backward of gated_linear_recurrence_fwd from its output h: returns
    (dx, dg, d(initial_state) or None), and d(gate_scale) as a fourth when
    `gate_scale` is given (dg is then the gradient of the logits)."""
    a = _abi_layer.gdn_linrec_bwd_args()
    _check("dh", dh)
    B, T, D, N, dev = _recurrence(a, dh, g, initial_state, cu_seqlens, gate_scale)
    _check("h", h, dh.dtype, (B, T, D), dev)
    _check("dht", dht, torch.float32, (N, D), dev)
    dx, dg = torch.empty_like(dh), torch.empty_like(dh)
    dh0 = torch.empty(N, D, dtype=torch.float32, device=dev) if want_dh0 else None
    a.d_h, a.h, a.d_final_state = dh.data_ptr(), h.data_ptr(), _ptr(dht)
    a.dx, a.dg, a.d_initial_state = dx.data_ptr(), dg.data_ptr(), _ptr(dh0)
    stream = _stream(dev)
    if gate_scale is None:
        _abi_layer.call_ws("gdn_linrec_bwd", a, 0, 0, stream)
        return dx, dg, dh0
    ds = torch.empty(D, dtype=torch.float32, device=dev)
    a.d_gate_scale = ds.data_ptr()
    n = _abi_layer.workspace_size("gdn_linrec_bwd", a)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _abi_layer.call_ws("gdn_linrec_bwd", a, ws.data_ptr(), n, stream)
    return dx, dg, dh0, ds


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
    a = _abi_layer.gdn_linrec_step_args()
    if x.dim() != 2:
        raise ValueError(f"expected [N, D] tensors, got shape {tuple(x.shape)}")
    a.dtype = _dtype("x", x)
    N, D = x.shape
    dev = x.device
    _check("x", x)
    _check("g", g, x.dtype, (N, D), dev)
    _check("state", state, torch.float32, (N, D), dev)
    _check("gate_scale", gate_scale, torch.float32, (D,), dev)
    _check("out_state", out_state, torch.float32, (N, D), dev)
    h = torch.empty_like(x)
    a.x, a.g, a.gate_scale, a.state = x.data_ptr(), g.data_ptr(), _ptr(gate_scale), state.data_ptr()
    a.N, a.D = N, D
    a.h, a.out_state = h.data_ptr(), state.data_ptr() if out_state is None else out_state.data_ptr()
    _abi_layer.call("gdn_linrec_step", a, _stream(dev))
    return h
