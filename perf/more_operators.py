"""The operators of a recurrent model's block that stand beside the delta rule, as cases to
measure: the short causal convolution and the selective state space scan behind it (forward,
backward, one token), and the gated feed-forward block (forward, backward).

`own` False: `run` computes them in elementary torch operations in 32 bits.
`own` True: `run` calls gated_deltanet_linear_bwd_gb300.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BLOCK = 512          # tokens that the plain scan takes at once


def _lib():
    import gated_deltanet_linear_bwd_gb300 as gdn
    return gdn


# ------------------------------------------------------------------ cases
def listed():
    """Widths are heads x head size of the package's workloads: 2 x 64 (tiny), 16 x 128 (long),
    32 x 128 (varlen, training)."""
    return [
        # ---- short causal convolution
        # one token for each of 64 running sequences: latency
        dict(name="conv_step", op="conv_step", N=64, D=4096, W=4, dtype="bf16", bias=True, silu=True),
        # a packed prefill batch of uneven requests
        dict(name="conv_fwd_varlen", op="conv_fwd", B=16, T=8192, D=4096, W=4, dtype="bf16", bias=True, silu=True,
             lo=512),
        # the training workload's backward pass
        dict(name="conv_bwd_train", op="conv_bwd", B=4, T=4096, D=4096, W=4, dtype="bf16", bias=True, silu=True,
             lo=0),
        # ---- selective state space scan
        # one token for each of 64 running sequences: latency, and the states' bytes
        dict(name="scan_step", op="scan_step", N=64, D=4096, S=16, dtype="bf16", logits=True, gate=True),
        # a unit-test-sized prefill of an odd length in full precision
        dict(name="scan_fwd_tiny", op="scan_fwd", B=1, T=257, D=128, S=16, dtype="fp32", logits=False, gate=False,
             lo=0),
        # one long document, few channels: the scan has to be split along the sequence
        dict(name="scan_fwd_long", op="scan_fwd", B=1, T=32768, D=2048, S=16, dtype="bf16", logits=True, gate=True,
             lo=0),
        # a packed prefill batch of uneven requests
        dict(name="scan_fwd_varlen", op="scan_fwd", B=16, T=4096, D=4096, S=16, dtype="bf16", logits=True, gate=True,
             lo=256),
        # a training step's backward pass
        dict(name="scan_bwd_train", op="scan_bwd", B=4, T=4096, D=2048, S=16, dtype="bf16", logits=True, gate=True,
             lo=0),
        # ---- gated feed-forward block
        # decode of 7 sequences: the weights' bytes bound it
        dict(name="ffn_decode", op="ffn_fwd", M=7, K=4096, F=12288, act="silu", save=False),
        # a ragged batch through a block of odd width, gelu
        dict(name="ffn_ragged", op="ffn_fwd", M=1000, K=2048, F=5464, act="gelu", save=False),
        # a training step's forward pass, keeping what the backward pass reads
        dict(name="ffn_fwd_train", op="ffn_fwd", M=8192, K=4096, F=12288, act="silu", save=True),
        # and its backward pass
        dict(name="ffn_bwd_train", op="ffn_bwd", M=8192, K=4096, F=12288, act="silu"),
    ]


def _size(rng, lo, hi, units=(1,)):
    """Spread over the logarithm of lo .. hi: an odd multiple of one of `units`, or a power of two."""
    n = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    if rng.random() < 0.3:
        return max(lo, 1 << int(math.log2(n) + 1e-9))
    unit = rng.choice(units)
    odd = 2 * int(n / (2 * unit)) + 1
    while odd > 1 and odd * unit > hi:
        odd -= 2
    return odd * unit


def draw(rng):
    op = rng.choice(["conv_step", "conv_fwd", "conv_bwd", "scan_step", "scan_fwd", "scan_fwd", "scan_bwd",
                     "ffn_fwd", "ffn_fwd", "ffn_bwd"])
    if op.startswith("ffn"):
        K, F = _size(rng, 64, 4096, (8, 64)), _size(rng, 64, 12288, (8, 64))
        M = _size(rng, 1, min(8192, (1 << 37) // (K * F)))
        c = dict(op=op, M=M, K=K, F=F, act=rng.choice(["silu", "silu", "gelu"]))
        return dict(c, save=rng.random() < 0.5) if op == "ffn_fwd" else c
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op.startswith("conv"):
        c.update(W=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.5, silu=rng.random() < 0.7)
    else:
        c.update(S=rng.choice([1, 5, 8, 16, 16, 16, 24, 64]), logits=rng.random() < 0.7, gate=rng.random() < 0.7)
    if op.endswith("step"):
        return dict(c, N=_size(rng, 1, 512), D=_size(rng, 1, 8192, (1, 2, 8)))
    B, D = _size(rng, 1, 16), _size(rng, 16, 4096, (1, 2, 8, 64))
    most = (1 << 26) // (B * D) if op == "conv_bwd" else (1 << 27) // (B * D) if op == "conv_fwd" else \
        (1 << (29 if op == "scan_bwd" else 30)) // (B * D * max(c["S"], 8))
    T = _size(rng, 1, max(1, min(65536 // B if op.startswith("scan") else 65536, most)))
    return dict(c, B=B, T=T, D=D, lo=T // 16 if rng.random() < 0.5 else 0)


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(c, seed):
    """Uneven request lengths of a packed batch, lo .. T each and one of them empty where lo is small:
    the same ones for a case, in the seed's order."""
    n = torch.randint(c["lo"], c["T"] + 1, (c["B"],), generator=torch.Generator().manual_seed(c["T"]))
    if c["lo"] < 64 and c["B"] > 2:
        n[1] = 0
    n[0] = max(1, int(n[0]))
    return n[torch.randperm(c["B"], generator=torch.Generator().manual_seed(seed))]


def _inputs(c, seed):
    gen = _generator(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def rand(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    op, i = c["op"], {}
    if op.startswith("ffn"):
        M, K, F = c["M"], c["K"], c["F"]
        i["x"] = randn(M, K).bfloat16()
        i["w_gate"], i["w_up"] = ((randn(F, K) * K ** -0.5).bfloat16() for _ in range(2))
        i["w_down"] = (randn(K, F) * F ** -0.5).bfloat16()
        if op == "ffn_bwd":
            # what a forward pass kept of normed tokens: of unit size
            i["gate"], i["up"], i["dy"] = randn(M, F).bfloat16(), randn(M, F).bfloat16(), randn(M, K).bfloat16()
        return i

    D, dt = c["D"], _DT[c["dtype"]]
    if op.endswith("step"):
        lead, N = (c["N"],), c["N"]
    elif c["lo"]:
        n = _lengths(c, seed)
        cu = torch.zeros(c["B"] + 1, dtype=torch.int32)
        cu[1:] = n.cumsum(0)
        i["cu"] = cu.cuda()
        lead, N = (1, int(cu[-1])), c["B"]
    else:
        lead, N = (c["B"], c["T"]), c["B"]
    i["x"] = randn(*lead, D).to(dt)
    if op.startswith("conv"):
        W = c["W"]
        i["w"] = (randn(D, W) * W ** -0.5).to(dt)
        if c["bias"]:
            i["bias"] = (0.1 * randn(D)).to(dt)
        i["h0"] = randn(N, W - 1, D).to(dt)
        if op == "conv_bwd":
            i["dy"], i["dht"] = randn(*lead, D).to(dt), (0.1 * randn(N, W - 1, D)).to(dt)
        return i

    S = c["S"]
    # the usual start of such a layer: a = -1 .. -S, steps spread over the logarithm of 0.001 .. 0.1
    i["a"] = -torch.arange(1, S + 1, device="cuda") * torch.exp(0.1 * randn(D, S))
    step = torch.exp(math.log(1e-3) + math.log(100.0) * rand(D))
    if c["logits"]:
        i["dt_bias"] = step + torch.log(-torch.expm1(-step))
        i["dt"] = (0.5 * randn(*lead, D)).to(dt)
    else:
        i["dt"] = (step * torch.exp(0.5 * randn(*lead, D))).to(dt)
    i["b"], i["c"] = randn(*lead, S).to(dt), randn(*lead, S).to(dt)
    i["skip"] = 1 + 0.1 * randn(D)
    if c["gate"]:
        i["z"] = randn(*lead, D).to(dt)
    i["h0"] = 0.1 * randn(N, D, S)
    if op == "scan_bwd":
        i["dy"], i["dht"] = randn(*lead, D).to(dt), 0.01 * randn(N, D, S)
    return i


def prepare(case, seed):
    return {"case": case, **_inputs(case, seed)}


# ------------------------------------------------------------------ plain forms
def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first dimension, by doubling the reach."""
    k, T = 1, a.shape[0]
    while k < T:
        b = torch.cat([b[:k], torch.addcmul(b[k:], a[k:], b[:-k])])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _ends(i, T, N):
    """First token, last token and length of each sequence, as indexes of flat tokens, and each token's sequence."""
    if "cu" in i:
        cu = i["cu"].long()
        t = torch.arange(T, device=cu.device)
        return cu[:-1], cu[1:] - 1, cu[1:] - cu[:-1], torch.searchsorted(cu[1:], t, right=True)
    t = torch.arange(N * T, device=i["x"].device)
    s = torch.arange(N, device=t.device) * T
    return s, s + T - 1, torch.full_like(s, T), t // T


def _conv_pre(i, x, first, seq):
    """Before the activation, and each tap's input."""
    W, bias = i["w"].shape[1], i.get("bias")
    w, h0 = i["w"].float(), i["h0"].float()
    local = torch.arange(x.shape[0], device=x.device) - first[seq]
    taps = []
    for k in range(W):
        back = local - (W - 1 - k)                     # the tap's place in its sequence, < 0: in the state
        shifted = x[(first[seq] + back).clamp(min=0)]
        early = (back < 0).nonzero()[:, 0]
        shifted[early] = h0[seq[early], W - 1 + back[early]]
        taps.append(shifted)
    pre = sum(w[:, k] * taps[k] for k in range(W))
    return (pre if bias is None else pre + bias.float()), taps


def _plain_conv(case, i):
    op, silu = case["op"], case["silu"]
    if op == "conv_step":
        xs = torch.cat([i["h0"], i["x"][:, None]], 1)
        pre = (xs.float() * i["w"].float().T).sum(1)
        pre = pre + i["bias"].float() if "bias" in i else pre
        return {"y": (pre * _sigmoid(pre) if silu else pre).to(i["x"].dtype), "state": xs[:, 1:].contiguous()}
    shape, D, W, dt = i["x"].shape, case["D"], case["W"], i["x"].dtype
    first, last, n, seq = _ends(i, shape[1], i["h0"].shape[0])
    x = i["x"].reshape(-1, D).float()
    pre, taps = _conv_pre(i, x, first, seq)
    if op == "conv_fwd":
        y = pre * _sigmoid(pre) if silu else pre
        # the last W - 1 inputs of state and sequence together
        at = n[:, None] - (W - 1) + torch.arange(W - 1, device=x.device)
        old = i["h0"].gather(1, (at + W - 1).clamp(0, W - 2)[..., None].expand(-1, -1, D))
        new = i["x"].reshape(-1, D)[(first[:, None] + at).clamp(0, x.shape[0] - 1)]
        return {"y": y.reshape(shape).to(dt), "state": torch.where((at >= 0)[..., None], new, old)}
    dpre = i["dy"].reshape(-1, D).float()
    if silu:
        s = _sigmoid(pre)
        dpre = dpre * s * (1 + pre * (1 - s))
    w, dht = i["w"].float(), i["dht"].float()
    local = torch.arange(x.shape[0], device=x.device) - first[seq]
    dx = torch.zeros_like(x)
    for k in range(W):                                 # token t is tap k of token t + W - 1 - k
        later = local + W - 1 - k
        inside = later < n[seq]
        dx += torch.where(inside[:, None], w[:, k] * dpre[(first[seq] + later).clamp(max=x.shape[0] - 1)], 0.0)
    tail = local + W - 1 - n[seq]                      # its place in the final state
    rows = (tail >= 0).nonzero()[:, 0]
    dx[rows] += dht[seq[rows], tail[rows]]
    dh0 = torch.zeros_like(dht)
    for j in range(W - 1):
        for k in range(j + 1):                         # the state's row j is tap k of token j - k
            inside = (j - k < n)[:, None]
            dh0[:, j] += torch.where(inside, w[:, k] * dpre[(first + j - k).clamp(max=x.shape[0] - 1)], 0.0)
        past = (j - n).clamp(min=0)
        dh0[:, j] += torch.where((j >= n)[:, None], dht.gather(1, past[:, None, None].expand(-1, 1, D))[:, 0], 0.0)
    out = {"dx": dx.reshape(shape).to(dt), "dw": torch.stack([(dpre * t).sum(0) for t in taps], 1),
           "dh0": dh0.to(dt)}
    if "bias" in i:
        out["dbias"] = dpre.sum(0)
    return out


def _steps(i):
    dt = i["dt"].float()
    return torch.nn.functional.softplus(dt + i["dt_bias"]) if "dt_bias" in i else dt


def _plain_scan(case, i):
    op, dt = case["op"], i["x"].dtype
    D, S = i["a"].shape
    if op == "scan_step":
        x, delta = i["x"].float(), _steps(i)
        h = torch.exp(delta[..., None] * i["a"]) * i["h0"] + (delta * x)[..., None] * i["b"].float()[:, None]
        y = (h * i["c"].float()[:, None]).sum(-1) + i["skip"] * x
        if "z" in i:
            z = i["z"].float()
            y = y * z * _sigmoid(z)
        return {"y": y.to(dt), "state": h}

    shape = i["x"].shape
    first, last, n, seq = _ends(i, shape[1], i["h0"].shape[0])
    x, delta = i["x"].reshape(-1, D).float(), _steps(i).reshape(-1, D)
    b, c = i["b"].reshape(-1, S).float(), i["c"].reshape(-1, S).float()
    T, h0 = x.shape[0], i["h0"]
    t = torch.arange(T, device=x.device)
    start, end = t == first[seq], t == last[seq]
    blocks = [slice(k, min(k + _BLOCK, T)) for k in range(0, T, _BLOCK)]

    def states(r, before):
        """Decays, inputs, states and each token's a h_{t-1} of tokens r, `before` the state ahead of them."""
        decay = torch.exp(delta[r][..., None] * i["a"])
        u = (delta[r] * x[r])[..., None] * b[r][:, None]
        rows = start[r].nonzero()[:, 0]
        a, v = decay.clone(), u.clone()
        v[0] += a[0] * before                           # overwritten below where a sequence begins
        v[rows] = u[rows] + decay[rows] * h0[seq[r][rows]]
        a[rows] = 0
        a[0] = 0
        return decay, u, _scan(a, v)

    ends, y = h0.clone(), torch.empty_like(x)
    before, kept = torch.zeros(D, S, device=x.device), []
    for r in blocks:
        kept.append(before)
        h = states(r, before)[2]
        before = h[-1]
        y[r] = (h * c[r][:, None]).sum(-1)
        rows = end[r].nonzero()[:, 0]
        ends[seq[r][rows]] = h[rows]
    s = y + i["skip"] * x
    if "z" in i:
        z = i["z"].reshape(-1, D).float()
        gate = z * _sigmoid(z)
    if op == "scan_fwd":
        y = s * gate if "z" in i else s
        return {"y": y.reshape(shape).to(dt), "state": ends}

    dy, out = i["dy"].reshape(-1, D).float(), {}
    ds = dy
    if "z" in i:
        ds = dy * gate
        out["dz"] = (dy * s * (_sigmoid(z) * (1 + z * (1 - _sigmoid(z))))).reshape(shape).to(dt)
    dx, ddelta, db, dc = i["skip"] * ds, torch.empty_like(x), torch.empty_like(b), torch.empty_like(c)
    da, dh0 = torch.zeros_like(i["a"]), i["dht"].clone()
    carry = torch.zeros(D, S, device=x.device)          # exp(delta a) e of the token after the block
    for r, before in zip(reversed(blocks), reversed(kept)):
        decay, u, h = states(r, before)
        e = ds[r][..., None] * c[r][:, None]
        rows = end[r].nonzero()[:, 0]
        nxt = torch.cat([decay[1:], decay[:1]])
        e[-1] += carry                                  # overwritten below where a sequence ends
        e[rows] = ds[r][rows][..., None] * c[r][rows][:, None] + i["dht"][seq[r][rows]]
        nxt[rows] = 0
        nxt[-1] = 0
        e = _scan(nxt.flip(0), e.flip(0)).flip(0)
        carry = decay[0] * e[0]
        rows = start[r].nonzero()[:, 0]
        dh0[seq[r][rows]] = decay[rows] * e[rows]
        prev = torch.cat([before[None], h[:-1]])
        prev[rows] = h0[seq[r][rows]]
        p = decay * prev
        dc[r] = (ds[r][..., None] * h).sum(1)
        db[r] = ((delta[r] * x[r])[..., None] * e).sum(1)
        eb, ep = (e * b[r][:, None]).sum(-1), e * p
        dx[r] += delta[r] * eb
        ddelta[r] = x[r] * eb + (ep * i["a"]).sum(-1)
        da += (delta[r][..., None] * ep).sum(0)
    out.update(dx=dx.reshape(shape).to(dt), da=da, db=db.reshape(*shape[:2], S).to(dt),
               dc=dc.reshape(*shape[:2], S).to(dt), dskip=(ds * x).sum(0), dh0=dh0)
    if "dt_bias" in i:
        ddelta = ddelta * _sigmoid(i["dt"].reshape(-1, D).float() + i["dt_bias"])
        out["ddt_bias"] = ddelta.sum(0)
    out["ddt"] = ddelta.reshape(shape).to(dt)
    return out


_GELU = math.sqrt(2 / math.pi)


def _activation(g, act):
    """The activation (gelu in its tanh form) and its derivative."""
    if act == "silu":
        s = _sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    s = _sigmoid(2 * _GELU * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * (1 - s) * 2 * _GELU * (1 + 3 * 0.044715 * g * g)


def _plain_ffn(case, i):
    x, wg, wu, wd = (i[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
    if case["op"] == "ffn_fwd":
        g, u = x @ wg.T, x @ wu.T
        y = (_activation(g, case["act"])[0] * u) @ wd.T
        out = {"y": y.bfloat16()}
        return dict(out, gate=g.bfloat16(), up=u.bfloat16()) if case["save"] else out
    g, u, dy = i["gate"].float(), i["up"].float(), i["dy"].float()
    f, slope = _activation(g, case["act"])
    dh = dy @ wd
    dg, du = dh * u * slope, dh * f
    return {"dx": (dg @ wg + du @ wu).bfloat16(), "dw_gate": (dg.T @ x).bfloat16(), "dw_up": (du.T @ x).bfloat16(),
            "dw_down": (dy.T @ (f * u)).bfloat16()}


# ------------------------------------------------------------------ one pass
def run(state):
    case, op = state["case"], state["case"]["op"]
    if not own:
        return (_plain_ffn if op.startswith("ffn") else _plain_conv if op.startswith("conv") else _plain_scan)(case, state)
    gdn, s = _lib(), state
    if op == "ffn_fwd":
        y, gate, up = gdn.gated_feed_forward_fwd(s["x"], s["w_gate"], s["w_up"], s["w_down"], activation=case["act"],
                                                 save=case["save"])
        return {"y": y, "gate": gate, "up": up} if case["save"] else {"y": y}
    if op == "ffn_bwd":
        out = gdn.gated_feed_forward_bwd(s["dy"], s["x"], s["w_gate"], s["w_up"], s["w_down"], s["gate"], s["up"],
                                         activation=case["act"])
        return dict(zip(("dx", "dw_gate", "dw_up", "dw_down"), out))
    if op.startswith("conv"):
        act = "silu" if case["silu"] else None
        if op == "conv_step":
            # the new state beside the old one, so that each pass starts from the same
            new = torch.empty_like(s["h0"])
            y = gdn.causal_convolution_step(s["x"], s["w"], s["h0"], bias=s.get("bias"), activation=act, out_state=new)
            return {"y": y, "state": new}
        if op == "conv_fwd":
            y, new = gdn.causal_convolution_fwd(s["x"], s["w"], bias=s.get("bias"), initial_state=s["h0"],
                                                cu_seqlens=s.get("cu"), activation=act)
            return {"y": y, "state": new}
        dx, dw, dbias, dh0 = gdn.causal_convolution_bwd(s["dy"], s["x"], s["w"], bias=s.get("bias"), dht=s["dht"],
                                                        initial_state=s["h0"], cu_seqlens=s.get("cu"), activation=act)
        out = {"dx": dx, "dw": dw, "dh0": dh0}
        return dict(out, dbias=dbias) if "bias" in s else out
    common = dict(skip=s["skip"], z=s.get("z"), dt_bias=s.get("dt_bias"))
    if op == "scan_step":
        new = torch.empty_like(s["h0"])
        y = gdn.state_space_step(s["x"], s["dt"], s["a"], s["b"], s["c"], s["h0"], out_state=new, **common)
        return {"y": y, "state": new}
    if op == "scan_fwd":
        y, new = gdn.state_space_scan_fwd(s["x"], s["dt"], s["a"], s["b"], s["c"], initial_state=s["h0"],
                                          cu_seqlens=s.get("cu"), **common)
        return {"y": y, "state": new}
    out = gdn.state_space_scan_bwd(s["dy"], s["x"], s["dt"], s["a"], s["b"], s["c"], dht=s["dht"],
                                   initial_state=s["h0"], cu_seqlens=s.get("cu"), **common)
    names = ("dx", "ddt", "da", "db", "dc", "dskip", "dz", "ddt_bias", "dh0")
    return {k: v for k, v in zip(names, out) if v is not None}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op.startswith("ffn"):
        M, K, F = case["M"], case["K"], case["F"]
        if op == "ffn_fwd":
            kept = 4 * M * F if case["save"] else 0
            return {"bytes": 4 * M * K + 6 * F * K + kept, "flops": 6.0 * M * F * K}
        return {"bytes": 6 * M * K + 4 * M * F + 12 * F * K, "flops": 12.0 * M * F * K}
    e, D = 2 if case["dtype"] == "bf16" else 4, case["D"]
    N = case["N"] if op.endswith("step") else case["B"]
    n = N if op.endswith("step") else N * ((case["lo"] + case["T"]) / 2 if case["lo"] else case["T"])   # tokens
    if op.startswith("conv"):
        W = case["W"]
        states, weight = 2 * e * N * (W - 1) * D, e * D * (W + 1)
        if op == "conv_bwd":
            return {"bytes": 3 * e * n * D + 1.5 * states + weight + 4 * D * (W + 1), "flops": (6.0 * W + 10) * n * D}
        return {"bytes": 2 * e * n * D + states + weight, "flops": (2.0 * W + 4) * n * D}
    S, gates = case["S"], 1 if case["gate"] else 0
    states, weight = 4 * N * D * S, 4 * D * (S + 2)
    if op == "scan_bwd":
        return {"bytes": e * n * (D * (5 + 2 * gates) + 4 * S) + 3 * states + 2 * weight, "flops": 25.0 * n * D * S}
    return {"bytes": e * n * (D * (3 + gates) + 2 * S) + 2 * states + weight, "flops": 7.0 * n * D * S}


# ------------------------------------------------------------------ the definitions in 64 bits
def _spans(case, i):
    if "cu" in i:
        cu = i["cu"].tolist()
        return list(zip(cu[:-1], cu[1:]))
    return [(n * case["T"], (n + 1) * case["T"]) for n in range(case["B"])]


def _exact_conv(case, i):
    W, D, silu = case["W"], case["D"], case["silu"]
    w, h0 = i["w"].double(), i["h0"].double()
    bias = i["bias"].double() if "bias" in i else 0.0
    if case["op"] == "conv_step":
        x = i["x"].double()
        pre = bias + w[:, W - 1] * x + sum(w[:, k] * h0[:, k] for k in range(W - 1))
        return {"y": pre * torch.special.expit(pre) if silu else pre,
                "state": torch.stack([h0[:, k] for k in range(1, W - 1)] + [x], 1)}
    x = i["x"].reshape(-1, D)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    states, dw, dbias = [], torch.zeros(W, D, dtype=torch.float64, device=x.device), 0.0
    for n, (a, b) in enumerate(_spans(case, i)):
        L, padded = b - a, torch.cat([h0[n], x[a:b].double()])
        pre = bias + sum(padded[k:k + L] * w[:, k] for k in range(W))
        if case["op"] == "conv_fwd":
            out[a:b] = pre * torch.special.expit(pre) if silu else pre
            states.append(padded[L:])
            continue
        dpre = i["dy"].reshape(-1, D)[a:b].double()
        if silu:
            sig = torch.special.expit(pre)
            dpre = dpre * (sig + pre * sig * (1 - sig))
        back = torch.zeros_like(padded)
        for k in range(W):
            back[k:k + L] += dpre * w[:, k]
            dw[k] += (dpre * padded[k:k + L]).sum(0)
        back[L:] += i["dht"][n].double()
        dbias = dbias + dpre.sum(0)
        out[a:b] = back[W - 1:]
        states.append(back[:W - 1])
    if case["op"] == "conv_fwd":
        return {"y": out.reshape(i["x"].shape), "state": torch.stack(states)}
    r = {"dx": out.reshape(i["x"].shape), "dw": dw.T.contiguous(), "dh0": torch.stack(states)}
    return dict(r, dbias=dbias) if "bias" in i else r


def _exact_scan(case, i):
    a, skip = i["a"].double(), i["skip"].double()
    D, S = a.shape

    def softplus(v):
        return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))

    if case["op"] == "scan_step":
        d = i["dt"].double()
        d = softplus(d + i["dt_bias"].double()) if "dt_bias" in i else d
        x = i["x"].double()
        h = torch.einsum("nd,ns->nds", d * x, i["b"].double()) + i["h0"].double() * torch.exp(torch.einsum("nd,ds->nds", d, a))
        y = torch.einsum("nds,ns->nd", h, i["c"].double()) + skip * x
        if "z" in i:
            y = y * i["z"].double() * torch.special.expit(i["z"].double())
        return {"y": y, "state": h}
    spans = _spans(case, i)
    if sum(q - p for p, q in spans) > 70_000:        # one token after another: too long a walk
        return None
    flat = {k: i[k].reshape(-1, i[k].shape[-1]) for k in ("x", "dt", "b", "c", "z", "dy") if k in i}
    back = case["op"] == "scan_bwd"
    new = lambda k: torch.empty(flat[k].shape, dtype=torch.float64, device=a.device)
    y, ends = new("x"), []
    g = {k: new(s) for k, s in (("dx", "x"), ("ddt", "dt"), ("db", "b"), ("dc", "c"))} if back else {}
    da, dskip, dbias, dh0, dz = torch.zeros_like(a), 0.0, 0.0, [], new("x")
    for n, (p, q) in enumerate(spans):
        L, now = q - p, i["h0"][n].double()
        v = {k: t[p:q].double() for k, t in flat.items()}
        raw = v["dt"] + (i["dt_bias"].double() if "dt_bias" in i else 0.0)
        d = softplus(raw) if "dt_bias" in i else raw
        hs = torch.empty(L + 1, D, S, dtype=torch.float64, device=a.device) if back else None
        if back:
            hs[0] = now
        dx = d * v["x"]
        for t in range(L):
            now = torch.exp(d[t, :, None] * a) * now + dx[t, :, None] * v["b"][t]
            y[p + t] = now @ v["c"][t]
            if back:
                hs[t + 1] = now
        ends.append(now)
        s = y[p:q] + skip * v["x"]
        gate = 1.0
        if "z" in v:
            sig = torch.special.expit(v["z"])
            gate = v["z"] * sig
        y[p:q] = s * gate
        if not back:
            continue
        ds = v["dy"] * gate
        if "z" in v:
            dz[p:q] = v["dy"] * s * (sig + v["z"] * sig * (1 - sig))
        carry = i["dht"][n].double()
        for t in range(L - 1, -1, -1):
            e = ds[t, :, None] * v["c"][t] + carry
            g["dc"][p + t] = ds[t] @ hs[t + 1]
            g["db"][p + t] = dx[t] @ e
            eb = e @ v["b"][t]
            carry = e * torch.exp(d[t, :, None] * a)
            lost = carry * hs[t]
            g["dx"][p + t] = skip * ds[t] + d[t] * eb
            g["ddt"][p + t] = v["x"][t] * eb + (lost * a).sum(-1)
            da += d[t, :, None] * lost
        dh0.append(carry)
        dskip = dskip + (ds * v["x"]).sum(0)
        if "dt_bias" in i:
            g["ddt"][p:q] *= torch.special.expit(raw)
            dbias = dbias + g["ddt"][p:q].sum(0)
    lead = i["x"].shape[:2]
    if not back:
        return {"y": y.reshape(i["x"].shape), "state": torch.stack(ends)}
    out = {k: t.reshape(*lead, -1) for k, t in g.items()}
    out.update(da=da, dskip=dskip, dh0=torch.stack(dh0))
    if "z" in i:
        out["dz"] = dz.reshape(i["x"].shape)
    return dict(out, ddt_bias=dbias) if "dt_bias" in i else out


def _exact_ffn(case, i):
    x, wg, wu, wd = (i[k].double() for k in ("x", "w_gate", "w_up", "w_down"))

    def act(g):
        if case["act"] == "silu":
            return g / (1 + torch.exp(-g))
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))

    if case["op"] == "ffn_fwd":
        g, u = torch.einsum("mk,fk->mf", x, wg), torch.einsum("mk,fk->mf", x, wu)
        out = {"y": torch.einsum("mf,kf->mk", act(g) * u, wd)}
        return dict(out, gate=g, up=u) if case["save"] else out
    g, u, dy = i["gate"].double(), i["up"].double(), i["dy"].double()
    if case["act"] == "silu":
        sig = torch.special.expit(g)
        slope = sig + g * sig * (1 - sig)
    else:
        th = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))
        slope = 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * math.sqrt(2 / math.pi) * (1 + 0.134145 * g * g)
    dh = torch.einsum("mk,kf->mf", dy, wd)
    dg, du = dh * u * slope, dh * act(g)
    return {"dx": torch.einsum("mf,fk->mk", dg, wg) + torch.einsum("mf,fk->mk", du, wu),
            "dw_gate": torch.einsum("mf,mk->fk", dg, x), "dw_up": torch.einsum("mf,mk->fk", du, x),
            "dw_down": torch.einsum("mk,mf->kf", dy, act(g) * u)}


def exact(case, seed):
    i, op = _inputs(case, seed), case["op"]
    return (_exact_ffn if op.startswith("ffn") else _exact_conv if op.startswith("conv") else _exact_scan)(case, i)
