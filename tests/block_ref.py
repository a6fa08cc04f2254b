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


def silu(z):
    return z * torch.sigmoid(z)


def silu_slope(z):
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def scan(x, dt, a, b, c, skip, z, dt_bias, h0, seqs):
    """x, dt, z [tokens, D], b, c [tokens, S], a [D, S], h0 [N, D, S]: (y, states)."""
    delta = dt if dt_bias is None else torch.nn.functional.softplus(dt + dt_bias, threshold=60)
    y, states = [], []
    for n, (p, q) in enumerate(seqs):
        h = h0[n]
        for t in range(p, q):
            h = torch.exp(delta[t, :, None] * a) * h + (delta[t] * x[t])[:, None] * b[t]
            y.append(h @ c[t])
        states.append(h)
    y = torch.stack(y) if y else torch.zeros_like(x)
    if skip is not None:
        y = y + skip * x
    return (y if z is None else y * silu(z)), torch.stack(states)


def scan_magnitudes(x, dt, a, b, c, skip, z, dt_bias, h0, dy, dht, seqs, signed=False):
    """What is summed in the scan and its gradients, every term by its magnitude (or, signed, as it is:
    then the results themselves), from the formulas: a dict."""
    m = (lambda t: t) if signed else torch.abs
    D, S = a.shape
    raw = dt if dt_bias is None else dt + dt_bias
    delta = dt if dt_bias is None else torch.nn.functional.softplus(raw, threshold=60)
    x, b, c, h0, dy, dht, step = m(x), m(b), m(c), m(h0), m(dy), m(dht), m(delta)
    skip = torch.zeros(D, dtype=torch.float64) if skip is None else m(skip)
    gate = torch.ones_like(x) if z is None else m(silu(z))
    ds = dy * gate
    out = {k: torch.zeros_like(v) for k, v in dict(y=x, dx=x, ddt=x, dz=x, db=b, dc=c, da=a, dh0=h0, state=h0).items()}
    decay = torch.exp(delta[..., None] * a)
    for n, (p, q) in enumerate(seqs):
        h, hs = h0[n], [h0[n]]
        for t in range(p, q):
            h = decay[t] * h + (step[t] * x[t])[:, None] * b[t]
            hs.append(h)
            out["y"][t] = h @ c[t] + skip * x[t]
        out["state"][n] = h
        e = dht[n]
        for t in range(q - 1, p - 1, -1):
            e = e + c[t] * ds[t][:, None]
            out["dc"][t] = ds[t] @ hs[t + 1 - p]
            out["db"][t] = (step[t] * x[t]) @ e
            out["dx"][t] = skip * ds[t] + step[t] * (e @ b[t])
            lost = e * decay[t] * hs[t - p]
            out["ddt"][t] = x[t] * (e @ b[t]) + (lost * m(a)).sum(1)
            out["da"] += lost * step[t][:, None]
            e = e * decay[t]
        out["dh0"][n] = e
    if z is not None:
        out["dz"] = dy * out["y"] * m(silu_slope(z))
        out["y"] = out["y"] * gate
    out["dskip"] = (ds * x).sum(0)
    if dt_bias is not None:
        out["ddt"] = out["ddt"] * torch.sigmoid(raw)
        out["ddt_bias"] = out["ddt"].sum(0)
    return out
