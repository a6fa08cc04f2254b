"""The selective state space scan on the GPU against 64 bits: forward, backward, one token."""
import pytest
import torch

from block_ref import HALF_STEP, inside, scan_magnitudes, spans
from gpu_helpers import lib

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
# A token multiplies the state by a decay that is off by 2^-22 (the exponential) and 2^-23 (its
# argument's roundings, at |delta a| < 4; softplus of a bf16 logit 2^-20 of delta, of which a decay
# sees delta a e^(delta a) < 0.4), and adds a product of three factors: 2^-20 of the magnitudes for
# each token that the state remembers, all T of them at most, and 2^-19 for what happens once.
TOKEN = 2.0 ** -20
ONCE = 2.0 ** -19
NAMES = ("dx", "ddt", "da", "db", "dc", "dskip", "dz", "ddt_bias", "dh0")


def make(dtype, B, T, D, S, cu=None, logits=True, gate=True, skip=True, state=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    N = B if cu is None else len(cu) - 1
    p = dict(x=r(B, T, D).to(dtype), dt=(r(B, T, D) - 1).to(dtype) if logits else (0.2 * r(B, T, D).abs()).to(dtype),
             a=-(torch.exp(r(D, S) - 1)).clamp(max=1.5).float(), b=r(B, T, S).to(dtype), c=r(B, T, S).to(dtype),
             skip=r(D).float() if skip else None, z=r(B, T, D).to(dtype) if gate else None,
             dt_bias=r(D).float() - 1 if logits else None)
    return dict(p=p, h0=r(N, D, S).float() if state else None, dy=r(B, T, D).to(dtype), dht=r(N, D, S).float(), cu=cu,
                N=N, seqs=spans(B, T, cu))


def gpu(t):
    return None if t is None else t.cuda()


def inputs(m):
    return {k: gpu(t) for k, t in m["p"].items()}


def cu_of(m):
    return None if m["cu"] is None else torch.tensor(m["cu"], dtype=torch.int32).cuda()


def reference(m, signed, dht=True):
    D, S = m["p"]["a"].shape
    flat = {k: None if t is None else t.double().reshape(-1, t.shape[-1]) if t.dim() == 3 else t.double()
            for k, t in m["p"].items()}
    zeros = torch.zeros(m["N"], D, S, dtype=torch.float64)
    h0 = zeros if m["h0"] is None else m["h0"].double()
    return scan_magnitudes(**flat, h0=h0, dy=m["dy"].double().reshape(-1, D), dht=m["dht"].double() if dht else zeros,
                           seqs=m["seqs"], signed=signed)


def check(m, got, dht=True):
    """Every output within what its rounding and the arithmetic of its terms allow."""
    want, size = reference(m, True, dht), reference(m, False, dht)
    longest = max([q - p for p, q in m["seqs"]], default=0)
    total = m["dy"].numel() // m["p"]["a"].shape[0]
    for k, t in got.items():
        if t is None:
            continue
        half = HALF_STEP[t.dtype]
        # sums over all tokens, and over the channels, besides the tokens of a state
        terms = total if k in ("da", "dskip", "ddt_bias") else m["p"]["a"].shape[0] if k in ("db", "dc") else 0
        bound = half * want[k].abs() * (1 + ONCE) + (ONCE + TOKEN * (longest + 1) + terms * 2.0 ** -24) * size[k]
        inside(k, t.reshape(want[k].shape), want[k], bound)


CU = [0, 1, 1, 3, 11, 75, 75, 76, 206]                    # lengths 1, 0, 2, 8, 64, 0, 1, 130
CASES = [
    # dtype, B, T, D, S, cu, logits, gate, skip, state
    (F, 1, 1, 1, 1, None, True, True, True, True),
    (F, 2, 9, 6, 3, None, False, False, False, False),
    (F, 2, 65, 33, 5, None, True, True, True, True),
    (F, 1, 206, 40, 16, CU, True, True, True, True),
    (F, 1, 129, 24, 17, None, False, True, False, True),
    (F, 1, 70, 9, 64, None, True, False, True, True),
    (BF, 1, 1, 8, 16, None, True, True, True, True),
    (BF, 3, 64, 72, 16, None, True, True, True, True),
    (BF, 2, 130, 264, 8, None, True, True, True, False),
    (BF, 1, 206, 130, 16, CU, True, True, True, True),
    (BF, 1, 206, 64, 4, CU, False, False, True, True),
    (BF, 1, 206, 520, 2, CU, True, True, False, True),
    (BF, 1, 206, 48, 32, CU, True, False, False, True),
    (BF, 1, 206, 24, 50, CU, True, True, True, True),
    (BF, 2, 300, 16, 64, None, False, True, True, True),
    (BF, 30, 3, 65, 16, None, True, True, True, True),
]


@pytest.mark.parametrize("dtype,B,T,D,S,cu,logits,gate,skip,state", CASES)
def test_forward_and_backward(dtype, B, T, D, S, cu, logits, gate, skip, state):
    gdn = lib()
    m = make(dtype, B, T, D, S, cu, logits, gate, skip, state)
    args = dict(initial_state=gpu(m["h0"]), cu_seqlens=cu_of(m), **inputs(m))
    y, ht = gdn.state_space_scan_fwd(**args)
    check(m, dict(y=y, state=ht))
    out = gdn.state_space_scan_bwd(gpu(m["dy"]), dht=gpu(m["dht"]), **args)
    assert [o is None for o in out] == [False] * 5 + [not skip, not gate, not logits, False]
    check(m, dict(zip(NAMES, out)))
    assert gdn.gdn_sync_status(0) == 0


@pytest.mark.parametrize("dtype,T,D,S", [(BF, 3000, 40, 16), (F, 2500, 12, 5), (BF, 2000, 8, 64)])
def test_sequences_cut_into_parts(dtype, T, D, S):
    """Few channels and a long sequence: walked in parts.  Long enough that a packed batch of it and
    short ones is too."""
    gdn = lib()
    for cu in (None, [0, 5, 5, T - 40, T]):
        m = make(dtype, 1, T, D, S, cu)
        n = gdn._abi_layer.ENTRIES["gdn_ssm_fwd"]
        assert n.workspace_size(n.pack(0, 0, 0, 0, 0, 0, 0, 0, 0, 16 if cu else 0, 1, T, D, S, m["N"],
                                       1 if dtype == BF else 0, 0, 0)) > 256
        args = dict(initial_state=gpu(m["h0"]), cu_seqlens=cu_of(m), **inputs(m))
        y, ht = gdn.state_space_scan_fwd(**args)
        check(m, dict(y=y, state=ht))
        check(m, dict(zip(NAMES, gdn.state_space_scan_bwd(gpu(m["dy"]), dht=gpu(m["dht"]), **args))))


@pytest.mark.parametrize("cu", [None, [0, 0, 0]])
def test_no_tokens_pass_the_state_on(cu):
    gdn = lib()
    m = make(BF, 1 if cu else 2, 0, 24, 16, cu)
    args = dict(initial_state=gpu(m["h0"]), cu_seqlens=cu_of(m), **inputs(m))
    y, ht = gdn.state_space_scan_fwd(**args)
    assert y.shape == m["dy"].shape and torch.equal(ht.cpu(), m["h0"])
    out = dict(zip(NAMES, gdn.state_space_scan_bwd(gpu(m["dy"]), dht=gpu(m["dht"]), **args)))
    assert torch.equal(out["dh0"].cpu(), m["dht"])
    assert not any(out[k].any() for k in ("da", "dskip", "ddt_bias"))


@pytest.mark.parametrize("dtype", [BF, F])
def test_steps_of_zero_keep_the_state_exactly(dtype):
    gdn = lib()
    m = make(dtype, 2, 50, 40, 16, logits=False)
    m["p"]["dt"].zero_()
    _, ht = gdn.state_space_scan_fwd(initial_state=gpu(m["h0"]), **inputs(m))
    assert torch.equal(ht.cpu(), m["h0"])


@pytest.mark.parametrize("dtype", [BF, F])
def test_slow_states_keep_their_size(dtype):
    """|delta a| of 0.0005 to 0.004 over 4096 steady tokens: each decay is within 2^-24 (its own
    rounding) and 1e-8 (what the hardware's exponential leans) of the true one, whatever the step."""
    gdn = lib()
    D, T = 64, 4096
    dt = torch.linspace(0.0005, 0.004, D).to(dtype)
    zeros = torch.zeros(1, T, D, dtype=dtype)
    one = torch.zeros(1, T, 1, dtype=dtype)
    _, ht = gdn.state_space_scan_fwd(zeros.cuda(), dt.expand(1, T, D).contiguous().cuda(), -torch.ones(D, 1).cuda(),
                                     one.cuda(), one.cuda(), initial_state=torch.ones(1, D, 1).cuda())
    want = torch.exp(-dt.double() * T)
    # two roundings of a token (the decay's and the product's), and the step's product with log2 e
    room = T * (2.0 ** -24 * 2 + 1.5e-8) + T * dt.double() * 2.0 ** -23
    inside("state", ht[0, :, 0], want, room * want)


@pytest.mark.parametrize("dtype,N,D,S", [(F, 1, 1, 1), (F, 5, 36, 6), (BF, 7, 72, 16), (BF, 64, 130, 64), (BF, 3, 33, 17)])
@pytest.mark.parametrize("logits", [True, False])
def test_steps_continue_a_prefill(dtype, N, D, S, logits):
    gdn = lib()
    m = make(dtype, N, 7, D, S, logits=logits)
    p = inputs(m)
    per_token = [k for k in ("x", "dt", "b", "c", "z")]
    want, size = reference(m, True), reference(m, False)
    part = {k: t[:, :4].contiguous() if k in per_token else t for k, t in p.items()}
    _, state = gdn.state_space_scan_fwd(initial_state=gpu(m["h0"]), **part)
    for t in range(4, 7):
        token = {k: v[:, t].clone() if k in per_token else v for k, v in p.items()}
        if t % 2:
            y = gdn.state_space_step(state=state, **token)
        else:
            new = torch.empty_like(state)
            y = gdn.state_space_step(state=state, out_state=new, **token)
            state = new
        w, s = (r["y"].view(N, 7, D)[:, t] for r in (want, size))
        inside("y", y, w, HALF_STEP[dtype] * w.abs() * (1 + ONCE) + (ONCE + 8 * TOKEN) * s)
    inside("state", state, want["state"], (ONCE + 8 * TOKEN) * size["state"])


def test_packed_sequences_are_separate_rows():
    """A packed sequence gives the bits of the same sequence alone (neither is cut into parts)."""
    gdn = lib()
    m = make(BF, 1, 206, 72, 16, CU)
    p = inputs(m)
    y, ht = gdn.state_space_scan_fwd(initial_state=gpu(m["h0"]), cu_seqlens=cu_of(m), **p)
    for n, (s, e) in enumerate(m["seqs"]):
        one = {k: t[:, s:e].clone() if t.dim() == 3 else t for k, t in p.items()}
        y1, h1 = gdn.state_space_scan_fwd(initial_state=gpu(m["h0"][n:n + 1].clone()), **one)
        assert torch.equal(y1, y[:, s:e]) and torch.equal(h1, ht[n:n + 1])


def test_many_sequences():
    """More than are put in the order of their length."""
    gdn = lib()
    gen = torch.Generator().manual_seed(4)
    lengths = torch.randint(0, 6, (300,), generator=gen).tolist()
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    m = make(BF, 1, cu[-1], 24, 8, cu)
    args = dict(initial_state=gpu(m["h0"]), cu_seqlens=cu_of(m), **inputs(m))
    y, ht = gdn.state_space_scan_fwd(**args)
    check(m, dict(y=y, state=ht))
    check(m, dict(zip(NAMES, gdn.state_space_scan_bwd(gpu(m["dy"]), dht=gpu(m["dht"]), **args))))


def test_a_nan_stays_in_its_channel_and_behind_its_token():
    gdn = lib()
    m = make(BF, 1, 40, 24, 16, [0, 20, 40], gate=False, skip=False)
    p = inputs(m)
    clean, _ = gdn.state_space_scan_fwd(cu_seqlens=cu_of(m), **p)
    p["x"][0, 7, 3] = float("nan")
    y, ht = gdn.state_space_scan_fwd(cu_seqlens=cu_of(m), **p)
    bad = torch.zeros(1, 40, 24, dtype=torch.bool)
    bad[0, 7:20, 3] = True
    assert torch.equal(torch.isnan(y).cpu(), bad)
    assert torch.equal(y.cpu()[~bad], clean.cpu()[~bad])
    assert torch.isnan(ht[0, 3]).all() and int(torch.isnan(ht).sum()) == 16


@pytest.mark.parametrize("cu", [[0, 5, 3, 40], [1, 20, 40], [0, 20, 39], [0, -7, 40], [0, 20, 2 ** 31 - 1], [0, 40, 40, 20, 40]])
def test_impossible_sequences_are_reported(cu):
    gdn = lib()
    m = make(BF, 1, 40, 16, 16)
    t = torch.tensor(cu, dtype=torch.int32).cuda()
    gdn.state_space_scan_fwd(cu_seqlens=t, **inputs(m))
    assert gdn.gdn_sync_status(0) == 6
    gdn.state_space_scan_bwd(gpu(m["dy"]), cu_seqlens=t, **inputs(m))
    assert gdn.gdn_sync_status(0) == 6
    assert gdn.gdn_sync_status(0) == 0


def test_gradients_against_differences():
    """Along a random direction, in fp32, with the third-order term of the difference taken out."""
    gdn = lib()
    m = make(F, 2, 40, 24, 8, seed=3)
    p = inputs(m)
    p["h0"] = gpu(m["h0"])
    gen = torch.Generator().manual_seed(9)
    way = {k: torch.randn(t.shape, generator=gen).cuda() for k, t in p.items()}
    dy, dht = gpu(m["dy"]), gpu(m["dht"])

    def loss(eps):
        v = {k: t + eps * way[k] for k, t in p.items()}
        y, ht = gdn.state_space_scan_fwd(initial_state=v.pop("h0"), **v)
        terms = torch.cat([(y.double() * dy.double()).flatten(), (ht.double() * dht.double()).flatten()])
        return float(terms.sum()), float(terms.abs().sum())

    eps = 2.0 ** -9
    (up, size), (down, _) = loss(eps), loss(-eps)
    (up2, _), (down2, _) = loss(2 * eps), loss(-2 * eps)
    d1, d2 = (up - down) / (2 * eps), (up2 - down2) / (4 * eps)
    slope = (4 * d1 - d2) / 3
    out = dict(zip(NAMES, gdn.state_space_scan_bwd(dy, dht=dht, initial_state=p["h0"],
                                                   **{k: t for k, t in p.items() if k != "h0"})))
    got = sum(float((out["d" + k].double() * way[k].double()).sum()) for k in p)
    # the losses' own error over the step (outputs within 40 TOKEN of their terms), and a tenth of the
    # third-order term for the fifth-order one
    assert abs(got - slope) <= 40 * TOKEN * size / eps + 0.1 * abs(d1 - d2)


def test_autograd():
    gdn = lib()
    m = make(BF, 1, 206, 72, 16, CU)
    leaves = {k: t.requires_grad_() for k, t in inputs(m).items()}
    h0 = gpu(m["h0"]).requires_grad_()
    y, ht = gdn.state_space_scan(**leaves, initial_state=h0, cu_seqlens=cu_of(m), output_final_state=True)
    got = torch.autograd.grad([y, ht], [*leaves.values(), h0], [gpu(m["dy"]), gpu(m["dht"])])
    plain = {k: t.detach() for k, t in leaves.items()}
    want = dict(zip(NAMES, gdn.state_space_scan_bwd(gpu(m["dy"]), dht=gpu(m["dht"]), initial_state=h0.detach(),
                                                    cu_seqlens=cu_of(m), **plain)))
    for k, g in zip([*leaves, "h0"], got):
        assert torch.equal(g, want["d" + k])
    # the loss of a slice, no gate and no states
    few = {k: leaves[k] for k in ("x", "dt", "a", "b", "c", "dt_bias")}
    y, none = gdn.state_space_scan(**few)
    assert none is None
    got = torch.autograd.grad(y[:, 1:3].sum(), list(few.values()))
    dy = torch.zeros_like(y)
    dy[:, 1:3] = 1
    want = dict(zip(NAMES, gdn.state_space_scan_bwd(dy, **{k: t.detach() for k, t in few.items()})))
    for k, g in zip(few, got):
        assert torch.equal(g, want["d" + k])


def test_captured_and_on_another_stream():
    gdn = lib()
    m = make(BF, 1, 2600, 40, 16, [0, 5, 2600])           # cut into parts
    args = dict(initial_state=gpu(m["h0"]), cu_seqlens=cu_of(m), **inputs(m))
    dy, dht = gpu(m["dy"]), gpu(m["dht"])

    def everything():
        return gdn.state_space_scan_fwd(**args) + gdn.state_space_scan_bwd(dy, dht=dht, **args)

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
    args["x"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, everything()))


def test_refusals():
    gdn = lib()
    m = make(BF, 2, 9, 16, 4)
    p = inputs(m)
    f = lambda **kw: gdn.state_space_scan_fwd(**{**p, **kw})
    for bad, word in [
        (lambda: f(x=p["x"][0]), "B, T, D"), (lambda: f(x=p["x"].half()), "dtype"), (lambda: f(dt=p["dt"].float()), "dt"),
        (lambda: f(a=p["a"].bfloat16()), "a must be"), (lambda: f(a=p["a"].repeat(1, 17)), "states"),
        (lambda: f(a=p["a"][:, :0]), "states"), (lambda: f(b=p["b"][:, :, :3].contiguous()), "b has shape"),
        (lambda: f(z=p["z"].cpu()), "z must be"), (lambda: f(skip=p["skip"].double()), "skip"),
        (lambda: f(dt_bias=p["dt_bias"][:8]), "dt_bias"), (lambda: f(initial_state=torch.zeros(2, 16, 5).cuda()), "shape"),
        (lambda: f(cu_seqlens=torch.zeros(2, 2, dtype=torch.int32).cuda()), "cu_seqlens"),
        (lambda: gdn.state_space_scan_bwd(gpu(m["dy"])[:1], **p), "shape"),
        (lambda: gdn.state_space_step(state=torch.zeros(2, 16, 4).cuda(), **p), "N, D"),
    ]:
        with pytest.raises(ValueError, match=word):
            bad()
    with pytest.raises(gdn.GdnError, match="cu_seqlens needs B == 1"):
        f(cu_seqlens=torch.tensor([0, 18], dtype=torch.int32).cuda())
