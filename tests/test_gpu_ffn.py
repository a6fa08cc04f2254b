"""The gated feed-forward block on the GPU against 64 bits: forward, backward."""
import pytest
import torch

from block_ref import HALF_STEP, inside
from gpu_helpers import lib

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HALF = HALF_STEP[BF]
# a sum of n products in the tensor cores' fp32: 2^-22 of the magnitudes for each addition (its rounding,
# or cutting off); activations and their slopes from the hardware's exponential: 2^-18
ADD, ARITH = 2.0 ** -22, 2.0 ** -18


def between(M, few):
    """What h, dg and du lose between the products: a rounding to bf16, or of few tokens at most two of them's."""
    return HALF if M > few else HALF * HALF


def make(M, K, F, seed=0, dtype=BF):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    return dict(x=r(M, K).to(dtype), w_gate=(r(F, K) * K ** -0.5).to(dtype), w_up=(r(F, K) * K ** -0.5).to(dtype),
                w_down=(r(K, F) * F ** -0.5).to(dtype), gate=r(M, F).to(dtype), up=r(M, F).to(dtype), dy=r(M, K).to(dtype))


def act(g, name):
    """The activation and its slope."""
    g = g.detach().clone().requires_grad_()
    f = g * torch.sigmoid(g) if name == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    return f.detach(), torch.autograd.grad(f.sum(), g)[0]


def gpu(p, *names):
    return [p[k].cuda() for k in names]


def close(name, got, want):
    """Independent roundings, two of them at most (an operand's, the result's), leave less of the norm
    than one's largest: each is 2^-8 / sqrt(3) on average."""
    d, n = (got.cpu().double() - want).norm(), want.norm()
    assert d <= HALF * n, f"{name}: off by {float(d / n):.2e} of its norm"


def check_forward(p, name, y, gate, up):
    x, wg, wu, wd = (p[k].double() for k in ("x", "w_gate", "w_up", "w_down"))
    K, F = wd.shape
    g, u = x @ wg.T, x @ wu.T
    eg, eu = (K * ADD * (x.abs() @ w.abs().T) for w in (wg, wu))
    if gate is not None:
        inside("gate", gate, g, HALF * (g.abs() + eg) + eg)
        inside("up", up, u, HALF * (u.abs() + eu) + eu)
    f, slope = act(g, name)
    h = f * u
    # the activation is off by eg times a slope of 1.13 at most
    eh = 1.13 * eg * (u.abs() + eu) + f.abs() * eu + ARITH * h.abs() + ARITH * 2.0 ** -6
    eh = eh + between(x.shape[0], 64) * (h.abs() + eh)
    want = h @ wd.T
    ey = eh @ wd.abs().T + F * ADD * ((h.abs() + eh) @ wd.abs().T)
    inside("y", y, want, ey + HALF * (want.abs() + ey))
    if want.numel() >= 64:
        close("y", y, want)


def check_backward(p, name, out):
    x, wg, wu, wd, g, u, dy = (p[k].double() for k in ("x", "w_gate", "w_up", "w_down", "gate", "up", "dy"))
    (K, F), M = wd.shape, x.shape[0]
    f, slope = act(g, name)
    dh = dy @ wd
    edh = K * ADD * (dy.abs() @ wd.abs())
    dg, du, h = dh * u * slope, dh * f, f * u
    # slopes of either activation are off by ARITH of 1 + |g|
    edg = edh * u.abs() * 1.13 + ARITH * (dh.abs() + edh) * u.abs() * (1 + g.abs())
    edu = edh * f.abs() + ARITH * (dh.abs() + edh) * (f.abs() + 2.0 ** -6)
    eh = ARITH * (h.abs() + 2.0 ** -6 * u.abs())
    edg, edu, eh = (e + between(M, 8) * (v.abs() + e) for e, v in ((edg, dg), (edu, du), (eh, h)))
    a = lambda t: t.abs()
    want = (dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ h)
    size = (a(dg) @ a(wg) + a(du) @ a(wu), a(dg).T @ a(x), a(du).T @ a(x), a(dy).T @ a(h))
    err = (edg @ a(wg) + edu @ a(wu), edg.T @ a(x), edu.T @ a(x), a(dy).T @ eh)
    for k, got, w, s, e, n in zip(("dx", "dw_gate", "dw_up", "dw_down"), out, want, size, err, (2 * F, M, M, M)):
        e = e + n * ADD * (s + e)
        inside(k, got, w, e + HALF * (a(w) + e))
        if w.numel() >= 64:
            close(k, got, w)


CASES = [(64, 520, 64, "gelu"), (65, 136, 200, "silu"), (8, 1200, 1032, "silu"), (9, 1200, 1032, "gelu"), (5, 2056, 136, "gelu"), (1, 8, 8, "silu"), (3, 64, 128, "gelu"), (7, 72, 136, "silu"), (16, 512, 264, "silu"), (33, 200, 520, "gelu"),
         (128, 128, 256, "silu"), (129, 264, 64, "gelu"), (257, 72, 392, "silu"), (300, 520, 1000, "silu"),
         (700, 256, 2048, "gelu"), (1, 1024, 4096, "silu"), (2500, 64, 72, "silu"),
         # wide enough for pairs of CTAs, into the block and out of it
         (2600, 72, 2000, "gelu"), (1300, 1928, 72, "silu")]


@pytest.mark.parametrize("M,K,F,name", CASES)
def test_forward(M, K, F, name):
    gdn = lib()
    p = make(M, K, F)
    args = gpu(p, "x", "w_gate", "w_up", "w_down")
    y, gate, up = gdn.gated_feed_forward_fwd(*args, activation=name, save=True)
    check_forward(p, name, y, gate, up)
    alone, none, _ = gdn.gated_feed_forward_fwd(*args, activation=name)
    assert none is None and torch.equal(alone, y)
    assert gdn.gdn_sync_status(0) == 0


@pytest.mark.parametrize("M,K,F,name", CASES)
def test_backward(M, K, F, name):
    gdn = lib()
    p = make(M, K, F)
    out = gdn.gated_feed_forward_bwd(*gpu(p, "dy", "x", "w_gate", "w_up", "w_down", "gate", "up"), activation=name)
    check_backward(p, name, out)
    assert gdn.gdn_sync_status(0) == 0


def test_more_tiles_than_the_gpu_has_pairs():
    """Several tiles to a pair of CTAs, with both accumulators in turn, ragged in every direction."""
    gdn = lib()
    p = make(1300, 136, 5000, seed=2)
    args = gpu(p, "x", "w_gate", "w_up", "w_down")
    y, gate, up = gdn.gated_feed_forward_fwd(*args, save=True)
    check_forward(p, "silu", y, gate, up)
    check_backward(p, "silu", gdn.gated_feed_forward_bwd(*gpu(p, "dy", "x", "w_gate", "w_up", "w_down", "gate", "up")))


def test_leading_dimensions_and_no_tokens():
    gdn = lib()
    p = make(12, 64, 128)
    x, wg, wu, wd, dy = gpu(p, "x", "w_gate", "w_up", "w_down", "dy")
    flat, gate, up = gdn.gated_feed_forward_fwd(x, wg, wu, wd, save=True)
    y, g3, u3 = gdn.gated_feed_forward_fwd(x.view(3, 4, 64), wg, wu, wd, save=True)
    assert y.shape == (3, 4, 64) and g3.shape == (3, 4, 128) and torch.equal(y.view(12, 64), flat)
    out = gdn.gated_feed_forward_bwd(dy.view(3, 4, 64), x.view(3, 4, 64), wg, wu, wd, g3, u3)
    for a, b in zip(out, gdn.gated_feed_forward_bwd(dy, x, wg, wu, wd, gate, up)):
        assert torch.equal(a.flatten(), b.flatten())
    y, gate, up = gdn.gated_feed_forward_fwd(x[:0], wg, wu, wd, save=True)
    assert y.shape == (0, 64) and gate.shape == (0, 128)
    dx, *dw = gdn.gated_feed_forward_bwd(dy[:0], x[:0], wg, wu, wd, gate, up)
    assert dx.shape == (0, 64) and not any(w.any() for w in dw)


@pytest.mark.parametrize("M", [3, 300])
def test_a_nan_stays_in_its_token(M):
    gdn = lib()
    p = make(M, 72, 136)
    x, wg, wu, wd = gpu(p, "x", "w_gate", "w_up", "w_down")
    clean = gdn.gated_feed_forward_fwd(x, wg, wu, wd)[0]
    x[1, 5] = float("nan")
    y = gdn.gated_feed_forward_fwd(x, wg, wu, wd)[0]
    assert torch.isnan(y[1]).all()
    keep = torch.arange(M) != 1
    assert torch.equal(y[keep], clean[keep])


def test_large_projections():
    """Activations far out: silu and gelu of +-200 are 200 and 0, their slopes 1 and 0."""
    gdn = lib()
    for name in ("silu", "gelu"):
        p = make(4, 64, 64)
        p["gate"] = torch.tensor([-200.0, 200.0, -1e4, 1e4] * 16).expand(4, 64).contiguous().to(BF)
        out = gdn.gated_feed_forward_bwd(*gpu(p, "dy", "x", "w_gate", "w_up", "w_down", "gate", "up"), activation=name)
        check_backward(p, name, out)


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gradients_against_differences(name):
    """Along a random direction: the gradient of the 64-bit block from differences of it, the block's own
    projections going in; bounded by the norm, as in close()."""
    gdn = lib()
    p = make(40, 64, 72, seed=5)
    names = ("x", "w_gate", "w_up", "w_down")
    leaves = [t.requires_grad_() for t in gpu(p, *names)]
    y = gdn.gated_feed_forward(*leaves, activation=name)
    grads = torch.autograd.grad(y, leaves, p["dy"].cuda())
    gen = torch.Generator().manual_seed(6)
    for k, grad in zip(names, grads):
        way = torch.randn(p[k].shape, generator=gen, dtype=torch.float64)
        way = way / way.norm()

        def loss(eps):
            v = {n: p[n].double() for n in names}
            v[k] = v[k] + eps * way
            h = act(v["x"] @ v["w_gate"].T, name)[0] * (v["x"] @ v["w_up"].T)
            return float(((h @ v["w_down"].T) * p["dy"].double()).sum())

        eps = 1e-4
        slope = (loss(eps) - loss(-eps)) / (2 * eps)
        # the projections' roundings come on top of the two of close(); on one direction of norm 1 the
        # whole gradient's error falls at most
        assert abs(float((grad.cpu().double() * way).sum()) - slope) <= 2 * HALF * float(grad.double().norm()) + 1e-5


def test_autograd():
    gdn = lib()
    p = make(50, 64, 136)
    leaves = [t.requires_grad_() for t in gpu(p, "x", "w_gate", "w_up", "w_down")]
    y = gdn.gated_feed_forward(*leaves, activation="gelu")
    dy = p["dy"].cuda()
    got = torch.autograd.grad(y, leaves, torch.cat([dy.flatten()[:1], dy.flatten()])[1:].view_as(dy))
    plain = [t.detach() for t in leaves]
    y2, gate, up = gdn.gated_feed_forward_fwd(*plain, activation="gelu", save=True)
    assert torch.equal(y, y2)
    for g, w in zip(got, gdn.gated_feed_forward_bwd(dy, *plain, gate, up, activation="gelu")):
        assert torch.equal(g, w)
    with torch.no_grad():
        assert torch.equal(gdn.gated_feed_forward(*leaves, activation="gelu"), y2)


@pytest.mark.parametrize("M", [5, 300])
def test_captured_and_on_another_stream(M):
    gdn = lib()
    p = make(M, 264, 520)
    args = gpu(p, "x", "w_gate", "w_up", "w_down")
    back = gpu(p, "dy", "x", "w_gate", "w_up", "w_down", "gate", "up")
    back[1] = args[0]

    def everything():
        return [t for t in gdn.gated_feed_forward_fwd(*args, save=True) + gdn.gated_feed_forward_bwd(*back)]

    want = everything()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = everything()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(g, w) for g, w in zip(there, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything()
    for t in got:
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    args[0].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, everything()))


@pytest.mark.parametrize("M", [5, 20, 600])
def test_waits_that_give_up_are_reported(M):
    """With a limit of no polls every wait gives up at once: the call returns, the status says so, and
    the next calls are whole again."""
    gdn = lib()
    p = make(M, 512, 1024)
    args = gpu(p, "x", "w_gate", "w_up", "w_down")
    back = gpu(p, "dy", "x", "w_gate", "w_up", "w_down", "gate", "up")
    gdn.gdn_set_spin_limit(0)
    try:
        gdn.gated_feed_forward_fwd(*args, save=True)
        assert gdn.gdn_sync_status(0) == 5
        gdn.gated_feed_forward_bwd(*back)
        assert gdn.gdn_sync_status(0) == (5 if M > 8 else 0)      # of so few tokens it has no waits
    finally:
        gdn.gdn_set_spin_limit(-1)
    y, gate, up = gdn.gated_feed_forward_fwd(*args, save=True)
    check_forward(p, "silu", y, gate, up)
    check_backward(p, "silu", gdn.gated_feed_forward_bwd(*back))
    assert gdn.gdn_sync_status(0) == 0


def test_refusals():
    gdn = lib()
    p = make(12, 64, 128)
    x, wg, wu, wd = gpu(p, "x", "w_gate", "w_up", "w_down")
    f = gdn.gated_feed_forward_fwd
    for bad, word in [
        (lambda: f(x.float(), wg, wu, wd), "bfloat16"), (lambda: f(x.half(), wg, wu, wd), "dtype"),
        (lambda: f(x, wg, wu, wd, activation="relu"), "activation"), (lambda: f(x, wg, wu, wd, activation=None), "activation"),
        (lambda: f(x, wg[0], wu, wd), "F, K"), (lambda: f(x, wg, wu[:64].contiguous(), wd), "w_up has shape"),
        (lambda: f(x, wg, wu, wd.T), "w_down"), (lambda: f(x, wg, wu, wg), "w_down has shape"),
        (lambda: f(x.cpu(), wg, wu, wd), "CUDA"), (lambda: f(x.T.contiguous().T, wg, wu, wd), "contiguous"),
        (lambda: gdn.gated_feed_forward_bwd(x, x, wg, wu, wd, wg, wg), "gate has shape"),
        (lambda: gdn.gated_feed_forward_bwd(x, x[:3], wg, wu, wd, wg, wg), "x has shape"),
    ]:
        with pytest.raises(ValueError, match=word):
            bad()
    odd = [torch.zeros(*s, dtype=BF, device="cuda") for s in ((3, 12), (8, 12), (8, 12), (12, 8))]
    with pytest.raises(gdn.GdnError, match="multiples of 8"):
        f(*odd)
