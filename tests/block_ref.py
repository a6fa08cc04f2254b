"""The short convolution, the state space scan and the gated feed-forward block in 64 bits, for the
tests: written from the formulas, one sequence and one token after another, apart from the library.
Gradients come from torch's differentiation of these."""
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}      # of a rounding, relative


def spans(B, T, cu):
    return [(n * T, (n + 1) * T) for n in range(B)] if cu is None else list(zip(cu[:-1], cu[1:]))


def convolution(x, w, bias, h0, seqs, silu):
    """x [tokens, D], w [D, W], h0 [N, W - 1, D]: (y, pre, states)."""
    W, pre, states = w.shape[1], [], []
    for n, (a, b) in enumerate(seqs):
        xp = torch.cat([h0[n], x[a:b]])
        p = sum(w[:, k] * xp[k:k + b - a] for k in range(W))
        pre.append(p if bias is None else p + bias)
        states.append(xp[b - a:])
    pre = torch.cat(pre)
    return pre * torch.sigmoid(pre) if silu else pre, pre, torch.stack(states)


def inside(name, got, want, bound):
    """Every element of got within `bound` of want."""
    got, want = got.detach().cpu().double(), want.detach()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if got.numel() == 0:
        return
    excess = (got - want).abs() - bound
    worst = excess.argmax()
    assert bool((excess <= 0).all()), (
        f"{name}: {int((excess > 0).sum())} of {got.numel()} out of bounds, worst {got.flatten()[worst]} for "
        f"{want.flatten()[worst]}, {float(excess.max()):.3e} past its bound")
