"""Infinite inputs of the state space block's operators: what the definitions give for them, and no
further than they reach."""
import pytest
import torch

from block_ref import HALF_STEP, convolution, inside, scan, scan_magnitudes
from gpu_helpers import lib
from test_gpu_ffn import ADD, gpu, make
from test_gpu_scan import ONCE, TOKEN

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
INF = float("inf")


# ------------------------------------------------------------------ feed-forward
@pytest.mark.parametrize("M", [3, 64, 65, 300])
def test_a_feature_that_overflows(M):
    """Feature 5 is 2^141 of token 1, and of token 2 3.402e38, which fp32 holds and bf16 rounds to infinity:
    however many tokens there are, the result is infinite, with the signs of its column of w_down."""
    gdn = lib()
    p = make(M, 72, 136)
    x, wg, wu, wd = gpu(p, "x", "w_gate", "w_up", "w_down")
    wg[:, 0], wu[:, 0] = 0, 0
    wd[:, 5] = torch.where(wd[:, 5] < 0, -0.5, 0.5)
    wg[5], wu[5] = 0, 0
    wg[5, 0], wu[5, 0] = 1, 2
    x[:, 0] = 0
    without = gdn.gated_feed_forward_fwd(x, wg, wu, wd)[0]
    x[1, 0], x[2, 0] = 2.0 ** 70, 181 / 128 * 2.0 ** 63
    y = gdn.gated_feed_forward_fwd(x, wg, wu, wd)[0]
    assert torch.isfinite(without).all()
    for t in (1, 2):
        assert torch.equal(y[t].float(), wd[:, 5].float() * INF)
    keep = torch.tensor([t for t in range(M) if t not in (1, 2)])
    assert torch.equal(y[keep], without[keep])


@pytest.mark.parametrize("M", [4, 300])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_slopes_of_the_largest_projections(M, name):
    """Gates whose square fp32 does not hold: the slope is 0 or 1."""
    gdn = lib()
    p = make(M, 64, 64)
    p["gate"] = torch.tensor([-1e20, 1e20, -3e38, 3e38, -2e19, 2e19, -1e30, 1e30] * 8).expand(M, 64).contiguous().to(BF)
    out = gdn.gated_feed_forward_bwd(*gpu(p, "dy", "x", "w_gate", "w_up", "w_down", "gate", "up"), activation=name)
    dy, wd, u, x = (p[k].double() for k in ("dy", "w_down", "up", "x"))
    on = (p["gate"] > 0).double()
    dg = (dy @ wd) * u * on
    edg = 64 * ADD * (dy.abs() @ wd.abs()) * u.abs() * on
    half = HALF_STEP[BF]
    edg = edg + half * (dg.abs() + edg)
    want = dg.T @ x
    e = edg.T @ x.abs() + M * ADD * ((dg.abs() + edg).T @ x.abs())
    inside("dw_gate", out[1], want, e + half * (want.abs() + e))


# ------------------------------------------------------------------ scan
def scan_inputs(dtype, T, D, S, skip, seed=0):
    """Positive coefficients, so that an infinite state is +inf and their sum is too."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    return dict(x=r(1, T, D).to(dtype), dt=(r(1, T, D) - 2).to(dtype), a=-torch.exp(r(D, S) - 2).float(),
                b=(r(1, T, S).abs() + 0.1).to(dtype), c=(r(1, T, S).abs() + 0.1).to(dtype),
                skip=(r(D).abs() + 0.1).float() if skip else None, z=r(1, T, D).to(dtype), dt_bias=r(D).float())


def on_gpu(p):
    return {k: None if t is None else t.cuda() for k, t in p.items()}


def definition(p, h0, T):
    flat = {k: None if t is None else t.double().reshape(-1, t.shape[-1]) if t.dim() == 3 else t.double()
            for k, t in p.items()}
    return scan(**flat, h0=h0.double(), seqs=[(0, T)])


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("S", [16, 64])
def test_an_infinite_input_without_skip(dtype, S):
    """With no skip nothing but the states takes x: they and the outputs are infinite from its token on."""
    gdn = lib()
    T, D = 40, 6
    p = scan_inputs(dtype, T, D, S, skip=False)
    clean, _ = gdn.state_space_scan_fwd(**on_gpu(p))
    p["x"][0, 7, 3], p["x"][0, 9, 4] = INF, -INF
    y, ht = gdn.state_space_scan_fwd(**on_gpu(p))
    want, state = definition(p, torch.zeros(1, D, S), T)
    assert want[7:, 3].isinf().all() and want[9:, 4].isinf().all()
    keep = want.isfinite()
    assert torch.equal(y[0].cpu()[keep], clean[0].cpu()[keep])
    assert torch.equal(y[0].cpu().double()[~keep], want[~keep])
    assert torch.equal(ht.cpu().isinf(), state.isinf()) and not torch.isnan(ht).any()
    # one token
    h0 = torch.rand(1, D, S)
    token = {k: t[:, 7].contiguous() if t is not None and t.dim() == 3 else t for k, t in p.items()}
    h = h0.cuda()
    y1 = gdn.state_space_step(state=h, **on_gpu(token))
    one = {k: t[:, 7:8] if t is not None and t.dim() == 3 else t for k, t in p.items()}
    want, state = definition(one, h0, 1)
    assert want[0, 3].isinf() and torch.equal(y1.cpu().double().isinf(), want.isinf()) and not torch.isnan(y1).any()
    assert torch.equal(h.cpu().isinf(), state.isinf()) and not torch.isnan(h).any()


@pytest.mark.parametrize("dtype", [BF, F])
def test_infinite_gradients_without_skip(dtype):
    """Nor does skip come into dz, which is infinite where the states are, and dx, from an infinite dy's
    token back."""
    gdn = lib()
    T, D, S = 40, 6, 16
    p = scan_inputs(dtype, T, D, S, skip=False)
    for k in ("b", "c", "z"):
        p[k] = p[k].abs() + 0.1
    dy = torch.ones(1, T, D, dtype=dtype)
    clean = gdn.state_space_scan_bwd(dy.cuda(), **on_gpu(p))
    p["x"][0, 7, 3] = INF
    dz = gdn.state_space_scan_bwd(dy.cuda(), **on_gpu(p))[6][0].cpu()
    bad = torch.zeros(T, D, dtype=torch.bool)
    bad[7:, 3] = True
    assert (dz[bad] == INF).all() and torch.equal(dz[~bad], clean[6][0].cpu()[~bad])
    p["x"][0, 7, 3] = 1
    clean = gdn.state_space_scan_bwd(dy.cuda(), **on_gpu(p))
    dy[0, 7, 3] = INF
    dx = gdn.state_space_scan_bwd(dy.cuda(), **on_gpu(p))[0][0].cpu()
    bad[:] = False
    bad[:8, 3] = True
    assert (dx[bad] == INF).all() and torch.equal(dx[~bad], clean[0][0].cpu()[~bad])


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("S", [1, 2, 3, 5, 8, 17, 24, 33, 50])
def test_infinities_with_any_number_of_states(dtype, S):
    """The lanes of a channel have places for more states than these: nothing comes of those, also where an
    input or a step (softplus of an infinite logit) is infinite; and the gradients are finite where the
    definition's are."""
    gdn = lib()
    T, D = 42, 6
    p = scan_inputs(dtype, T, D, S, skip=True)
    p["x"][0, 7, 3], p["x"][0, 9, 4], p["dt"][0, 20, 1] = INF, -INF, INF
    y, ht = gdn.state_space_scan_fwd(**on_gpu(p))
    zeros = torch.zeros(1, D, S)
    want, state = definition(p, zeros, T)
    assert int(want.isinf().sum()) == 35 + 33 + 22 and not torch.isnan(want).any()
    infinite = want.isinf()
    assert torch.equal(y[0].cpu().isinf(), infinite) and not torch.isnan(y).any()
    assert torch.equal(y[0].cpu().double()[infinite], want[infinite])
    assert torch.equal(ht.cpu().double()[state.isinf()], state[state.isinf()]) and not torch.isnan(ht).any()
    for t in (7, 9, 20):
        token = {k: v[:, t].contiguous() if v.dim() == 3 else v for k, v in p.items()}
        h = torch.ones(1, D, S).cuda()
        y1 = gdn.state_space_step(state=h, **on_gpu(token))
        want, state = definition({k: v[:, t:t + 1] if v.dim() == 3 else v for k, v in p.items()}, zeros + 1, 1)
        assert torch.equal(y1.cpu().isinf(), want.isinf()) and not torch.isnan(y1).any()
        assert torch.equal(h.cpu().isinf(), state.isinf()) and not torch.isnan(h).any()
    dy, dht = torch.ones(1, T, D, dtype=dtype), torch.ones(1, D, S)
    flat = {k: v.double().reshape(-1, v.shape[-1]) if v.dim() == 3 else v.double() for k, v in p.items()}
    want = scan_magnitudes(**flat, h0=zeros.double(), dy=dy[0].double(), dht=dht.double(), seqs=[(0, T)], signed=True)
    out = gdn.state_space_scan_bwd(dy.cuda(), dht=dht.cuda(), **on_gpu(p))
    for k, t in zip(("dx", "ddt", "da", "db", "dc", "dskip", "dz", "ddt_bias", "dh0"), out):
        assert torch.isfinite(t.reshape(want[k].shape).cpu()[want[k].isfinite()]).all(), k


@pytest.mark.parametrize("dtype", [BF, F])
def test_an_infinite_state_of_a_sequence_cut_into_parts(dtype):
    """A part's decay underflows (32 steps of 1.5 times a = -2 and less), which no token's does: the state
    stays infinite to the end."""
    gdn = lib()
    T, D, S = 3000, 6, 5
    p = scan_inputs(dtype, T, D, S, skip=True)
    p["a"] = -2 - torch.rand(D, S, generator=torch.Generator().manual_seed(1))
    p["dt"], p["dt_bias"] = torch.full((1, T, D), 1.5, dtype=dtype), None
    n = gdn._abi_layer.ENTRIES["gdn_ssm_fwd"]
    assert n.workspace_size(n.pack(*[0] * 10, 1, T, D, S, 1, 1 if dtype == BF else 0, 0, 0)) > 256
    clean, ht0 = gdn.state_space_scan_fwd(**on_gpu(p))
    p["x"][0, 500, 3], p["x"][0, 2, 4] = INF, -INF
    y, ht = gdn.state_space_scan_fwd(**on_gpu(p))
    want, state = definition(p, torch.zeros(1, D, S), T)
    assert int(want.isinf().sum()) == 2500 + 2998 and int(state.isinf().sum()) == 2 * S
    keep = want.isfinite()
    assert torch.equal(y[0].cpu()[keep], clean[0].cpu()[keep]) and torch.equal(y[0].cpu().double()[~keep], want[~keep])
    keep = state.isfinite()
    assert torch.equal(ht.cpu()[keep], ht0.cpu()[keep]) and torch.equal(ht.cpu().double()[~keep], state[~keep])


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [1, 33, 42, 63])
def test_the_last_input_infinite(dtype, T):
    """Nothing comes after it: a's gradient, which takes the states before each token, stays finite."""
    gdn = lib()
    D, S = 6, 16
    p = scan_inputs(dtype, T, D, S, skip=False)
    dy, dht, h0 = torch.ones(1, T, D, dtype=dtype).cuda(), torch.ones(1, D, S).cuda(), torch.ones(1, D, S).cuda()
    clean = gdn.state_space_scan_bwd(dy, dht=dht, initial_state=h0, **on_gpu(p))
    p["x"][0, T - 1, 3] = INF
    out = gdn.state_space_scan_bwd(dy, dht=dht, initial_state=h0, **on_gpu(p))
    for k, i in (("dx", 0), ("da", 2), ("dh0", 8)):
        assert torch.equal(out[i], clean[i]), k


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("S", [5, 16])
def test_masked_steps(dtype, S):
    """A logit of -inf is a step of zero: the states pass such tokens as they are, whatever their finite x, and
    the gradients are those of the sequence without them."""
    gdn = lib()
    T, D = 50, 10
    p = scan_inputs(dtype, T, D, S, skip=True)
    for k in ("b", "c"):
        p[k] = p[k] - 0.5
    masked = torch.zeros(T, dtype=torch.bool)
    masked[[0, 3, 4, 5, 17, 31, 32, 48, 49]] = True
    p["dt"][0, masked] = -INF
    p["x"][0, masked] = 1e30
    h0, dht = torch.ones(1, D, S).cuda(), torch.ones(1, D, S).cuda()
    dy = torch.randn(1, T, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    dy[0, masked] = 0
    few = {k: t[:, ~masked].contiguous() if t.dim() == 3 else t for k, t in p.items()}
    y, ht = gdn.state_space_scan_fwd(initial_state=h0, **on_gpu(p))
    y2, ht2 = gdn.state_space_scan_fwd(initial_state=h0, **on_gpu(few))
    assert torch.equal(ht, ht2) and torch.equal(y[:, ~masked], y2) and torch.isfinite(y).all()
    out = gdn.state_space_scan_bwd(dy.cuda(), dht=dht, initial_state=h0, **on_gpu(p))
    assert not out[0][0, masked].any() and not out[1][0, masked].any()
    flat = {k: t.double().reshape(-1, t.shape[-1]) if t.dim() == 3 else t.double() for k, t in few.items()}
    want, size = (scan_magnitudes(**flat, h0=h0.cpu().double(), dy=dy[0, ~masked].double(), dht=dht.cpu().double(),
                                  seqs=[(0, len(dy[0, ~masked]))], signed=signed) for signed in (True, False))
    for k, g in zip(("dx", "ddt", "da", "db", "dc", "dskip", "dz", "ddt_bias", "dh0"), out):
        g = g[:, ~masked] if g.dim() == 3 and k != "dh0" else g
        # as test_gpu_scan's check: a result's rounding, and what its terms lose token by token
        room = HALF_STEP[g.dtype] * want[k].abs() * (1 + ONCE) + (ONCE + TOKEN * (T + 1) + T * 2.0 ** -24) * size[k]
        inside(k, g.reshape(want[k].shape), want[k], room)


# ------------------------------------------------------------------ convolution
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("D", [7, 264])
def test_an_infinity_stays_under_its_taps(dtype, silu, D):
    gdn = lib()
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen)
    T, W, cu = 40, 4, torch.tensor([0, 9, 40], dtype=torch.int32).cuda()
    x, w, b, dy = r(1, T, D).to(dtype), r(D, W).to(dtype), r(D).to(dtype), r(1, T, D).to(dtype).cuda()
    act = "silu" if silu else None
    run = lambda: (gdn.causal_convolution_fwd(x.cuda(), w.cuda(), b.cuda(), cu_seqlens=cu, activation=act),
                   gdn.causal_convolution_bwd(dy, x.cuda(), w.cuda(), b.cuda(), cu_seqlens=cu, activation=act))
    (y0, h0), (dx0, dw0, db0, dh0) = run()
    x[0, 7, 3], x[0, 20, 5] = INF, -INF
    (y1, h1), (dx1, dw1, db1, dh1) = run()
    want, _, state = convolution(x[0].double(), w.double(), b.double(), torch.zeros(2, W - 1, D, dtype=torch.float64),
                                 [(0, 9), (9, 40)], silu)
    y0, y1, dx0, dx1 = (t[0].cpu() for t in (y0, y1, dx0, dx1))
    keep = want.isfinite()
    assert int((~keep).sum()) == 2 + 4 and torch.equal(y1[keep], y0[keep])
    assert torch.equal(torch.isnan(y1), torch.isnan(want)) and torch.equal(y1[y1.isinf()].double(), want[want.isinf()])
    assert torch.equal(h1.cpu().double(), state)
    # dx of the tokens whose outputs the infinity reaches (with silu, whose slope there is NaN), and its channels'
    # sums
    reach = torch.zeros(T, D, dtype=torch.bool)
    if silu:
        reach[4:9, 3], reach[17:24, 5] = True, True
    assert torch.equal(dx1[~reach], dx0[~reach]) and not torch.isfinite(dx1[reach]).any()
    others = torch.tensor([d for d in range(D) if d not in (3, 5)])
    assert torch.equal(dw1[others], dw0[others]) and torch.equal(db1[others], db0[others]) and torch.equal(dh1, dh0)
    assert not torch.isfinite(dw1[5]).any()
