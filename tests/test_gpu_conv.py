"""The short causal convolution on the GPU against 64 bits: forward, backward, one token."""
import pytest
import torch

from block_ref import HALF_STEP, convolution, inside, spans
from gpu_helpers import lib

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
# fp32 arithmetic: the taps' sums (at most 5 terms), and for bf16 tensors the hardware's exponential
# and reciprocal, off by 2^-21 each: 2^-19 of the magnitudes that enter covers a product of a few
ARITH = 2.0 ** -19


def make(dtype, B, T, D, W, cu=None, bias=True, state=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64).to(dtype)
    N = B if cu is None else len(cu) - 1
    return dict(x=r(B, T, D), w=r(D, W), bias=r(D) if bias else None, h0=r(N, W - 1, D) if state else None,
                dy=r(B, T, D), dht=r(N, W - 1, D), cu=cu, N=N, seqs=spans(B, T, cu))


def gpu(t):
    return None if t is None else t.cuda()


def cu_of(p):
    return None if p["cu"] is None else torch.tensor(p["cu"], dtype=torch.int32).cuda()


def reference(p, silu, dht=True):
    D, W = p["w"].shape
    leaf = lambda t: t.double().requires_grad_()
    x, w = leaf(p["x"].reshape(-1, D)), leaf(p["w"])
    bias = leaf(p["bias"]) if p["bias"] is not None else None
    h0 = leaf(p["h0"]) if p["h0"] is not None else torch.zeros(p["N"], W - 1, D, dtype=torch.float64, requires_grad=True)
    y, pre, ht = convolution(x, w, bias, h0, p["seqs"], silu)
    pre.retain_grad()
    loss = (y * p["dy"].reshape(-1, D).double()).sum() + ((ht * p["dht"].double()).sum() if dht else 0.0)
    loss.backward()
    # what enters each sum, for the bounds
    mag = convolution(x.abs(), w.abs(), None if bias is None else bias.abs(), h0.abs(), p["seqs"], False)[1].detach()
    return dict(x=x, w=w, bias=bias, h0=h0, y=y, pre=pre, ht=ht, mag=mag)


def check_forward(p, y, ht, r):
    D = p["w"].shape[0]
    half = HALF_STEP[p["x"].dtype]
    inside("y", y.reshape(-1, D), r["y"], half * r["y"].abs() * (1 + ARITH) + ARITH * r["mag"])
    if ht is not None:
        assert torch.equal(ht.cpu().double(), r["ht"].detach())        # inputs, moved


def check_backward(p, out, r, silu):
    dx, dw, db, dh0 = out
    D, W = p["w"].shape
    half = HALF_STEP[p["x"].dtype]
    dy = p["dy"].reshape(-1, D).double().abs()
    # dpre = dy (s + pre s (1 - s)): off by ARITH of dy (1 + pre), and by what pre is off times the
    # slope's own slope (at most 0.5)
    off = (ARITH * dy * (1 + r["pre"].abs() + r["mag"])).detach() if silu else torch.zeros_like(dy)
    g = r["pre"].grad.abs()
    xa, wa = r["x"].detach().abs(), r["w"].detach().abs()
    ref = lambda dpre: through(p, dpre, wa, xa, r["h0"].detach().abs())
    sx, sw, sb, sh = ref(g)                               # magnitudes that are summed
    ox, ow, ob, oh = ref(off)                             # their errors
    n = dy.shape[0] + 64                                  # a sum of n terms in any order: n 2^-24 of them
    inside("dx", dx.reshape(-1, D), r["x"].grad, half * r["x"].grad.abs() * (1 + ARITH) + ARITH * sx + ox)
    inside("dw", dw, r["w"].grad, n * 2.0 ** -24 * sw + ow)
    if db is not None:
        inside("db", db, r["bias"].grad, n * 2.0 ** -24 * sb + ob)
    if dh0 is not None:
        inside("dh0", dh0, r["h0"].grad, half * r["h0"].grad.abs() * (1 + ARITH) + ARITH * sh + oh)


def through(p, dpre, w, x, h0):
    """dx, dw, db, dh0 of the linear part, of magnitudes."""
    x, w, h0 = (t.clone().requires_grad_() for t in (x, w, h0))
    b = torch.zeros(w.shape[0], dtype=torch.float64, requires_grad=True)
    _, pre, ht = convolution(x, w, b, h0, p["seqs"], False)
    ((pre * dpre).sum() + (ht * p["dht"].double().abs()).sum()).backward()
    return x.grad, w.grad, b.grad, h0.grad


CU = [0, 1, 1, 3, 6, 46, 46, 200]                         # lengths 1, 0, 2, 3, 40, 0, 154
CASES = [
    # dtype, B, T, D, W, cu, silu, bias, state
    (F, 1, 1, 1, 2, None, True, True, True),
    (F, 2, 5, 6, 3, None, True, False, True),
    (F, 3, 100, 130, 4, None, False, True, False),
    (F, 1, 200, 12, 4, CU, True, True, True),
    (BF, 1, 1, 8, 4, None, True, True, True),
    (BF, 2, 2, 5, 4, None, True, True, True),            # rows shorter than the taps
    (BF, 2, 33, 24, 4, None, True, True, True),
    (BF, 1, 700, 264, 2, None, True, False, False),
    (BF, 3, 65, 1026, 3, None, False, True, True),
    (BF, 1, 200, 72, 4, CU, True, True, True),
    (BF, 1, 200, 33, 3, CU, True, False, False),
    (BF, 1, 200, 2064, 4, CU, False, True, True),
    (BF, 40, 1, 16, 4, None, True, True, True),           # rows of one token
]


@pytest.mark.parametrize("dtype,B,T,D,W,cu,silu,bias,state", CASES)
def test_forward_and_backward(dtype, B, T, D, W, cu, silu, bias, state):
    gdn = lib()
    p = make(dtype, B, T, D, W, cu, bias, state)
    act = "silu" if silu else None
    r = reference(p, silu)
    args = dict(bias=gpu(p["bias"]), initial_state=gpu(p["h0"]), cu_seqlens=cu_of(p), activation=act)
    y, ht = gdn.causal_convolution_fwd(gpu(p["x"]), gpu(p["w"]), **args)
    check_forward(p, y, ht, r)
    out = gdn.causal_convolution_bwd(gpu(p["dy"]), gpu(p["x"]), gpu(p["w"]), dht=gpu(p["dht"]), **args)
    check_backward(p, out, r, silu)
    assert gdn.gdn_sync_status(0) == 0


@pytest.mark.parametrize("dtype", [F, BF])
def test_without_states(dtype):
    gdn = lib()
    p = make(dtype, 2, 37, 40, 4, state=False)
    r = reference(p, True, dht=False)
    y, ht = gdn.causal_convolution_fwd(gpu(p["x"]), gpu(p["w"]), bias=gpu(p["bias"]), output_final_state=False)
    assert ht is None
    check_forward(p, y, None, r)
    dx, dw, db, dh0 = gdn.causal_convolution_bwd(gpu(p["dy"]), gpu(p["x"]), gpu(p["w"]), bias=gpu(p["bias"]), want_dh0=False)
    assert dh0 is None
    p["dht"] = torch.zeros_like(p["dht"])
    check_backward(p, (dx, dw, db, None), r, True)


@pytest.mark.parametrize("cu", [None, [0, 0, 0]])
def test_no_tokens_pass_the_state_on(cu):
    gdn = lib()
    p = make(BF, 1 if cu else 2, 0, 24, 4, cu)
    args = dict(bias=gpu(p["bias"]), initial_state=gpu(p["h0"]), cu_seqlens=cu_of(p))
    y, ht = gdn.causal_convolution_fwd(gpu(p["x"]), gpu(p["w"]), **args)
    assert y.shape == p["x"].shape and torch.equal(ht.cpu(), p["h0"])
    dx, dw, db, dh0 = gdn.causal_convolution_bwd(gpu(p["dy"]), gpu(p["x"]), gpu(p["w"]), dht=gpu(p["dht"]), **args)
    assert torch.equal(dh0.cpu(), p["dht"]) and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype,N,D,W", [(F, 1, 1, 2), (F, 5, 36, 3), (BF, 7, 72, 4), (BF, 64, 1030, 4), (BF, 3, 33, 2)])
@pytest.mark.parametrize("act", ["silu", None])
def test_steps_continue_a_prefill(dtype, N, D, W, act):
    """Steps from a prefill's state give the bits of the forward pass over all tokens."""
    gdn = lib()
    p = make(dtype, N, 9, D, W)
    x, w, b, h0 = (gpu(p[k]) for k in ("x", "w", "bias", "h0"))
    whole, last = gdn.causal_convolution_fwd(x, w, b, h0, activation=act)
    _, state = gdn.causal_convolution_fwd(x[:, :5].contiguous(), w, b, h0, activation=act)
    for t in range(5, 9):
        if t % 2:
            y = gdn.causal_convolution_step(x[:, t].clone(), w, state, b, act)
        else:
            new = torch.empty_like(state)
            y = gdn.causal_convolution_step(x[:, t].clone(), w, state, b, act, out_state=new)
            state = new
        assert torch.equal(y, whole[:, t])
    assert torch.equal(state, last)


def test_packed_sequences_are_separate_rows():
    gdn = lib()
    p = make(BF, 1, 200, 72, 4, CU)
    x, w, b, h0 = (gpu(p[k]) for k in ("x", "w", "bias", "h0"))
    y, ht = gdn.causal_convolution_fwd(x, w, b, h0, cu_of(p))
    for n, (s, e) in enumerate(p["seqs"]):
        if e > s:
            one, h = gdn.causal_convolution_fwd(x[:, s:e].contiguous(), w, b, h0[n:n + 1].contiguous())
            assert torch.equal(one, y[:, s:e]) and torch.equal(h, ht[n:n + 1])


def test_infinite_and_nan_inputs_stay_in_their_reach():
    """A NaN reaches the W tokens whose taps see it, in its own channel and sequence."""
    gdn = lib()
    p = make(BF, 1, 40, 16, 4, [0, 20, 40])
    x, w = gpu(p["x"]), gpu(p["w"])
    clean, _ = gdn.causal_convolution_fwd(x, w, cu_seqlens=cu_of(p))
    x[0, 18, 3] = float("nan")
    y, ht = gdn.causal_convolution_fwd(x, w, cu_seqlens=cu_of(p))
    bad = torch.zeros(1, 40, 16, dtype=torch.bool)
    bad[0, 18:20, 3] = True
    assert torch.equal(torch.isnan(y).cpu(), bad)
    assert torch.equal(y.cpu()[~bad], clean.cpu()[~bad])
    assert torch.isnan(ht[0, 1, 3]) and int(torch.isnan(ht).sum()) == 1


@pytest.mark.parametrize("cu", [[0, 5, 3, 40], [1, 20, 40], [0, 20, 39], [0, -7, 40], [0, 20, 2 ** 31 - 1]])
def test_impossible_sequences_are_reported(cu):
    gdn = lib()
    p = make(BF, 1, 40, 16, 4)
    N = len(cu) - 1
    t = torch.tensor(cu, dtype=torch.int32).cuda()
    h0 = torch.zeros(N, 3, 16, dtype=BF).cuda()
    gdn.causal_convolution_fwd(gpu(p["x"]), gpu(p["w"]), initial_state=h0, cu_seqlens=t)
    assert gdn.gdn_sync_status(0) == 6
    gdn.causal_convolution_bwd(gpu(p["dy"]), gpu(p["x"]), gpu(p["w"]), initial_state=h0, dht=h0, cu_seqlens=t)
    assert gdn.gdn_sync_status(0) == 6
    assert gdn.gdn_sync_status(0) == 0


def test_gradients_against_differences():
    """Along a random direction, in fp32: the difference's own error is that of its two losses (2^-24
    of the sum of |y dy|, times 4 for y's arithmetic) over the step, and its third-order term."""
    gdn = lib()
    p = make(F, 2, 50, 24, 4, seed=3)
    names = ("x", "w", "bias", "h0")
    at = [gpu(p[k]) for k in names]
    gen = torch.Generator().manual_seed(9)
    way = [torch.randn(t.shape, generator=gen).cuda() for t in at]
    dy, dht = gpu(p["dy"]), gpu(p["dht"])

    def loss(eps):
        y, ht = gdn.causal_convolution_fwd(*(t + eps * d for t, d in zip(at, way)))
        return (y.double() * dy.double()).sum() + (ht.double() * dht.double()).sum(), (y.double() * dy.double()).abs().sum()

    eps = 2.0 ** -7
    (up, size), (down, _) = loss(eps), loss(-eps)
    (up2, _), (down2, _) = loss(2 * eps), loss(-2 * eps)
    d1, d2 = (up - down) / (2 * eps), (up2 - down2) / (4 * eps)
    slope = (4 * d1 - d2) / 3                              # the third-order term taken out
    dx, dw, db, dh0 = gdn.causal_convolution_bwd(dy, at[0], at[1], at[2], dht, at[3])
    got = sum((g.double() * d.double()).sum() for g, d in zip((dx, dw, db, dh0), way))
    room = float(size) * 2.0 ** -22 / eps + float((d1 - d2).abs()) * 4 * eps + 1e-5 * float(size)
    assert abs(float(got - slope)) <= room


def test_autograd():
    gdn = lib()
    p = make(BF, 1, 200, 72, 4, CU)
    leaves = [gpu(p[k]).requires_grad_() for k in ("x", "w", "bias", "h0")]
    y, ht = gdn.causal_convolution(*leaves[:3], initial_state=leaves[3], cu_seqlens=cu_of(p), output_final_state=True)
    got = torch.autograd.grad([y, ht], leaves, [gpu(p["dy"]), gpu(p["dht"])])
    want = gdn.causal_convolution_bwd(gpu(p["dy"]), *(t.detach() for t in leaves[:3]), gpu(p["dht"]), leaves[3].detach(),
                                      cu_of(p))
    for g, w, leaf in zip(got, want, leaves):
        assert g.dtype == leaf.dtype and torch.equal(g, w.to(leaf.dtype))
    # gradients that are slices, on no 16-byte boundary; no final state; no bias
    x, w = (gpu(p[k]).requires_grad_() for k in ("x", "w"))
    y, none = gdn.causal_convolution(x, w, cu_seqlens=cu_of(p), activation=None)
    assert none is None
    dy = torch.cat([gpu(p["dy"]).flatten()[:1], gpu(p["dy"]).flatten()])[1:].view_as(y)
    got = torch.autograd.grad(y, (x, w), dy)
    want = gdn.causal_convolution_bwd(gpu(p["dy"]), x.detach(), w.detach(), cu_seqlens=cu_of(p), activation=None)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1].to(BF))


def test_captured_and_on_another_stream():
    gdn = lib()
    p = make(BF, 1, 200, 72, 4, CU)
    x, w, b, h0, dy, dht = (gpu(p[k]) for k in ("x", "w", "bias", "h0", "dy", "dht"))
    cu = cu_of(p)

    def both():
        return gdn.causal_convolution_fwd(x, w, b, h0, cu) + gdn.causal_convolution_bwd(dy, x, w, b, dht, h0, cu)

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(g, w) for g, w in zip(there, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for t in got:
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, both()))


def test_refusals():
    gdn = lib()
    p = make(BF, 2, 9, 16, 4)
    x, w, h0 = gpu(p["x"]), gpu(p["w"]), gpu(p["h0"])
    f = gdn.causal_convolution_fwd
    for bad, word in [
        (lambda: f(x[0], w), "B, T, D"), (lambda: f(x.double(), w), "dtype"), (lambda: f(x.cpu(), w), "CUDA"),
        (lambda: f(x.transpose(0, 1), w), "contiguous"), (lambda: f(x, w.float()), "bfloat16"),
        (lambda: f(x, w[:, :1].contiguous()), "taps"), (lambda: f(x, torch.cat([w, w], 1)), "taps"),
        (lambda: f(x, w[:8].contiguous()), "shape"), (lambda: f(x, w, activation="gelu"), "activation"),
        (lambda: f(x, w, initial_state=h0[:, :2].contiguous()), "shape"), (lambda: f(x, w, bias=w[:, 0]), "bias"),
        (lambda: f(x, w, cu_seqlens=torch.zeros(1, dtype=torch.int32).cuda()), "cu_seqlens"),
        (lambda: f(x, w, cu_seqlens=torch.zeros(3).cuda()), "int32"),
        (lambda: gdn.causal_convolution_step(x[:, 0].contiguous(), w, h0.float()), "state"),
        (lambda: gdn.causal_convolution_bwd(gpu(p["dy"]), x[:1].contiguous(), w), "shape"),
    ]:
        with pytest.raises(ValueError, match=word):
            bad()
    with pytest.raises(gdn.GdnError, match="cu_seqlens needs B == 1"):
        f(x, w, cu_seqlens=torch.tensor([0, 18], dtype=torch.int32).cuda())
    with pytest.raises(gdn.GdnError, match="aligned"):
        f(torch.zeros(2 * 9 * 16 + 1, dtype=BF, device="cuda")[1:].view(2, 9, 16), w)
