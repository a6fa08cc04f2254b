"""The per-channel gated linear recurrence against its definition in 64 bits:
forward, backward and step, fp32 and bf16, log decays and gate logits, lengths
from none to many tiles, odd widths, packed batches with empty sequences,
resets and infinite gates, more than 2^31 elements, other streams, refusals.

Tolerances.  u = 2^-24.  A token's decay carries at most c u relative error:
c = 8 covers expf (2 ulp), the product and the sum of its step and the same
again for the pairs' composition; with bf16 gate logits the hardware logarithm
and exponential add at most 3e-7 (5 u) to softplus, hence 8 u |gate_scale| to
the log decay: c = 16.  The error of a state then follows E_t = a_t E_{t-1} +
c u m_t with m_t = a_t m_{t-1} + |x_t|, computed beside the reference.  Outputs
stored in bf16, of 8 significant bits, add 2^-8 of their own magnitude."""
import numpy as np
import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def log_decay(g, scale):
    return g if scale is None else -scale * (np.maximum(g, 0) + np.log1p(np.exp(-np.abs(g))))


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


class Problem:
    def __init__(self, B, T, D, dtype, gated, h0=True, lengths=None, seed=0):
        gen = torch.Generator().manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=gen)
        self.lengths = [T] * B if lengths is None else lengths
        if lengths is not None:
            B, T = 1, sum(lengths)
        self.N, dt = len(self.lengths), DT[dtype]
        self.dtype, self.cu = dtype, None
        if lengths is not None:
            self.cu = torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32).cuda()
        a = torch.rand(D, generator=gen) * 0.99 + 0.01
        self.x, self.dh = randn(B, T, D).to(dt).cuda(), randn(B, T, D).to(dt).cuda()
        z = randn(B, T, D)
        self.scale = a.cuda() if gated else None
        self.g = (z if gated else -torch.nn.functional.softplus(z) * a).to(dt).cuda()
        self.h0 = randn(self.N, D).cuda() if h0 else None
        self.dht = randn(self.N, D).cuda() if h0 else None
        self.c = (16 if gated and dtype == "bf16" else 8) * U

    def spans(self):
        ends = np.cumsum([0] + self.lengths)
        return list(zip(ends[:-1], ends[1:]))

    def flat(self, t):
        return np64(t).reshape(-1, t.shape[-1])


def reference_fwd(p):
    x, l = p.flat(p.x), log_decay(p.flat(p.g), np64(p.scale))
    D = x.shape[1]
    h, E = np.zeros_like(x), np.zeros_like(x)
    ht, Et = np.zeros((p.N, D)), np.zeros((p.N, D))
    for n, (lo, hi) in enumerate(p.spans()):
        now = np64(p.h0)[n].copy() if p.h0 is not None else np.zeros(D)
        m, e = np.abs(now), np.zeros(D)
        for t in range(lo, hi):
            a = np.exp(l[t])
            now = a * now + x[t]
            m = a * m + np.abs(x[t])
            e = a * e + p.c * m
            h[t], E[t] = now, e
        ht[n], Et[n] = now, e
    return h, E, ht, Et


def reference_bwd(p, h):
    dh, g = p.flat(p.dh), p.flat(p.g)
    scale = np64(p.scale)
    l, h = log_decay(g, scale), p.flat(h)
    D = dh.shape[1]
    out = {k: np.zeros_like(dh) for k in ("dx", "dl")}
    err = {k: np.zeros_like(dh) for k in ("dx", "dl")}
    dh0, E0 = np.zeros((p.N, D)), np.zeros((p.N, D))
    for n, (lo, hi) in enumerate(p.spans()):
        c = np64(p.dht)[n].copy() if p.dht is not None else np.zeros(D)
        m, e = np.abs(c), np.zeros(D)
        for t in range(hi - 1, lo - 1, -1):
            a = np.exp(l[t])
            hp = h[t - 1] if t > lo else (np64(p.h0)[n] if p.h0 is not None else np.zeros(D))
            d = dh[t] + c
            m = m + np.abs(dh[t])
            e = e + p.c * m
            out["dx"][t], err["dx"][t] = d, e
            c, m, e = a * d, a * m, a * (e + p.c * m)
            out["dl"][t], err["dl"][t] = c * hp, (e + p.c * np.abs(c)) * np.abs(hp)
        dh0[n], E0[n] = c, e
    out["dh0"], err["dh0"] = dh0, E0
    dl, edl = out.pop("dl"), err.pop("dl")
    if scale is None:
        out["dg"], err["dg"] = dl, edl
    else:
        sp = np.maximum(g, 0) + np.log1p(np.exp(-np.abs(g)))
        sig = 0.5 * (1 + np.tanh(g / 2))
        out["dg"], err["dg"] = -scale * sig * dl, scale * sig * (edl + p.c * np.abs(dl))
        # a sum of T terms: each one's error, and the sum's own (T roundings of partial sums,
        # bounded by the sum of magnitudes)
        out["ds"] = -(sp * dl).sum(0)
        err["ds"] = (sp * edl + 4 * p.c * (sp + 1) * np.abs(dl)).sum(0) + \
            U * 64 * np.abs(sp * dl).sum(0)
    return out, err


def close(name, got, want, err, dtype):
    got = np64(got).reshape(want.shape)
    tol = err + 1e-30
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(want) + 1e-38
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (name, int(bad.sum()), float(np.abs(got - want)[bad].max()), float(tol[bad].min()))


CASES = [
    # B, T, D, lengths
    (1, 1, 1, None), (2, 0, 8, None), (3, 1, 64, None), (1, 17, 63, None), (2, 128, 64, None),
    (1, 129, 130, None), (1, 1000, 33, None), (2, 2500, 256, None), (1, 9001, 40, None),
    (0, 0, 96, [5, 0, 300, 1, 0]), (0, 0, 45, [0, 0, 700]), (0, 0, 512, [1] * 40),
    (0, 0, 64, [0]), (0, 0, 2, [3000, 4, 129]),
    # long enough to be cut into parts: TMA rows, plain ones, packed with short and empty ones beside
    (1, 40000, 64, None), (2, 30001, 24, None), (1, 33000, 9, None), (0, 0, 32, [50000, 0, 100, 20, 40000]),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("B,T,D,lengths", CASES)
def test_forward_and_backward_match_the_definition(B, T, D, lengths, gated, dtype):
    for h0 in (True, False):
        p = Problem(B, T, D, dtype, gated, h0=h0, lengths=lengths, seed=T + D)
        h, ht = lib().gated_linear_recurrence_fwd(p.x, p.g, p.h0, p.cu, p.scale)
        want, E, want_t, Et = reference_fwd(p)
        close("h", h, want, E, dtype)
        close("final state", ht, want_t, Et, "fp32")
        got = lib().gated_linear_recurrence_bwd(p.dh, p.g, h, p.dht, p.h0, p.cu, p.scale)
        out, err = reference_bwd(p, h)
        for name, t in zip(("dx", "dg", "dh0", "ds"), got):
            close(name, t, out[name], err[name], dtype if name in ("dx", "dg") else "fp32")
        assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 64), (5, 33), (64, 4096), (0, 16)])
def test_steps_continue_the_recurrence(N, D, gated, dtype):
    p = Problem(max(N, 1), 4, D, dtype, gated, seed=N + D)
    state, want = p.h0[:N].contiguous(), np64(p.h0[:N])
    err = np.zeros_like(want)
    for t in range(4):
        x, g = (v[:N, t].clone() for v in (p.x, p.g))
        h = lib().gated_linear_recurrence_step(x, g, state, p.scale)
        a = np.exp(log_decay(np64(g), np64(p.scale)))
        err = a * err + p.c * (a * np.abs(want) + np.abs(np64(x)))
        want = a * want + np64(x)
        close("h", h, want, err, dtype)
        close("state", state, want, err, "fp32")
    if N:
        other = torch.full_like(state, float("nan"))
        before = state.clone()
        lib().gated_linear_recurrence_step(x, g, state, p.scale, out_state=other)
        assert torch.equal(state, before) and torch.isfinite(other).all()


def test_gradients_match_central_differences():
    """In fp32 on inputs of a few tokens: the derivative of sum(h * dh) + sum(ht * dht) along random
    directions.  Step 1e-2: the third-order term and the rounding of a sum of ~100 terms of size ~1
    (100 * 2^-24 / 1e-2 = 6e-4) both stay below 3e-3 of the derivative's scale."""
    gen = torch.Generator().manual_seed(3)
    x, g, dh = (torch.randn(1, 9, 6, generator=gen).cuda() for _ in range(3))
    s, h0, dht = torch.rand(6, generator=gen).cuda() + 0.1, torch.randn(2, 6, generator=gen).cuda(), \
        torch.randn(2, 6, generator=gen).cuda()
    cu = torch.tensor([0, 4, 9], dtype=torch.int32).cuda()
    ins = [t.requires_grad_() for t in (x, g, h0, s)]

    def f(x, g, h0, s):
        h, ht = lib().gated_linear_recurrence(x, g, h0, cu, s, output_final_state=True)
        return (h.double() * dh).sum() + (ht.double() * dht).sum()

    grads = torch.autograd.grad(f(*ins), ins)
    for k, grad in enumerate(grads):
        d = torch.randn(grad.shape, generator=gen).cuda()
        with torch.no_grad():
            up, down = ([t + sign * 1e-2 * d if j == k else t for j, t in enumerate(ins)]
                        for sign in (1, -1))
            num = float((f(*up) - f(*down)) / 2e-2)
        want = float((grad.double() * d).sum())
        scale = float(grad.double().norm() * d.double().norm())
        assert abs(num - want) <= 3e-3 * scale, (k, num, want, scale)


@pytest.mark.parametrize("gated", [False, True])
def test_resets_and_infinite_gates(gated):
    """A log decay of -inf (a gate logit of +inf) forgets everything before it; a logit of -inf
    keeps the state as it is."""
    for dtype in ("fp32", "bf16"):
        p = Problem(1, 400, 64, dtype, gated, seed=1)
        p.g[0, ::37] = float("inf") if gated else float("-inf")
        if gated:
            p.g[0, 100:105] = float("-inf")
        with np.errstate(all="ignore"):
            want, E, want_t, Et = reference_fwd(p)
        h, ht = lib().gated_linear_recurrence_fwd(p.x, p.g, p.h0, None, p.scale)
        close("h", h, want, E, dtype)
        close("ht", ht, want_t, Et, "fp32")
        dx, dg, dh0 = lib().gated_linear_recurrence_bwd(p.dh, p.g, h, p.dht, p.h0, None, p.scale)[:3]
        assert torch.equal(dg[0, ::37], torch.zeros_like(dg[0, ::37]))
        assert torch.isfinite(dx).all() and torch.isfinite(dh0).all()


def test_nan_stays_in_its_channel_and_its_sequence():
    p = Problem(0, 0, 66, "bf16", True, lengths=[200, 50], seed=2)
    p.g[0, 70, 5] = float("nan")
    h, ht = lib().gated_linear_recurrence_fwd(p.x, p.g, p.h0, p.cu, p.scale)
    bad = torch.isnan(h[0])
    want = torch.zeros_like(bad)
    want[70:200, 5] = True
    assert torch.equal(bad, want)
    assert torch.isnan(ht).sum() == 1 and torch.isnan(ht[0, 5])


def test_more_than_2_to_31_elements():
    """B T D = 2.2e9: the last row alone has to equal the last row of the batch."""
    B, T, D = 67, 8192, 4096
    x = torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda").normal_()
    g = torch.empty_like(x).normal_()
    s = torch.rand(D, device="cuda")
    h, ht = lib().gated_linear_recurrence_fwd(x, g, None, None, s)
    h1, ht1 = lib().gated_linear_recurrence_fwd(x[-1:].contiguous(), g[-1:].contiguous(), None, None, s)
    a = torch.exp(-s.double() * torch.nn.functional.softplus(g[-1, -1].double()))
    before = a * h1[0, -2].double()
    last = before + x[-1, -1].double()
    assert ((h[-1, -1].double() - last).abs() <= 2.0 ** -8 * (last.abs() + before.abs())).all()
    assert (h[-1].float() - h1[0].float()).abs().max() <= 2.0 ** -7 * h1.float().abs().max()
    assert torch.allclose(ht[-1], ht1[0], rtol=1e-4, atol=1e-4)


def test_repeats_bit_for_bit_and_on_another_stream():
    p = Problem(1, 5000, 192, "bf16", True, seed=4)
    run = lambda: (*lib().gated_linear_recurrence_fwd(p.x, p.g, p.h0, None, p.scale),
                   *lib().gated_linear_recurrence_bwd(p.dh, p.g, p.x, p.dht, p.h0, None, p.scale))
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(side):
            again = run()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_bad_cu_seqlens_is_recorded_and_the_next_call_is_right():
    p = Problem(0, 0, 64, "fp32", False, lengths=[30, 20], seed=5)
    for bad in ([0, 60, 50], [1, 30, 50], [0, 30, 49], [0, -4, 50]):
        cu = torch.tensor(bad, dtype=torch.int32).cuda()
        lib().gated_linear_recurrence_fwd(p.x, p.g, p.h0, cu, p.scale)
        assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 6
    h, ht = lib().gated_linear_recurrence_fwd(p.x, p.g, p.h0, p.cu, p.scale)
    want, E, want_t, Et = reference_fwd(p)
    close("h", h, want, E, "fp32")
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0


def test_refusals():
    p = Problem(2, 8, 64, "bf16", True)
    f, b, s = (getattr(lib(), "gated_linear_recurrence_" + k) for k in ("fwd", "bwd", "step"))
    one = p.x[:, 0].contiguous()
    for bad in (lambda: f(p.x.cpu(), p.g), lambda: f(p.x, p.g.float()), lambda: f(p.x.half(), p.g.half()),
                lambda: f(p.x[..., ::2], p.g[..., ::2]), lambda: f(p.x, p.g[:, :4].contiguous()),
                lambda: f(p.x, p.g, p.h0[:1]), lambda: f(p.x, p.g, p.h0.bfloat16()),
                lambda: f(p.x, p.g, None, torch.tensor([0, 8], device="cuda")),
                lambda: f(p.x, p.g, None, None, p.scale[:3].contiguous()), lambda: f(p.x[0], p.g[0]),
                lambda: b(p.dh, p.g, p.x.float()), lambda: b(p.dh, p.g, p.x, p.dht[:1]),
                lambda: s(one, one, p.h0[:, :3].contiguous()), lambda: s(p.x, p.g, p.h0),
                lambda: s(one, one, p.h0, out_state=p.h0.bfloat16())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lib().GdnError, match="cu_seqlens"):     # packed tokens come as one row
        f(p.x, p.g, None, torch.tensor([0, 8, 16], dtype=torch.int32).cuda())
    with pytest.raises(lib().GdnError, match="aligned"):
        odd = torch.empty(1 + 2 * 8 * 64, dtype=torch.bfloat16, device="cuda")[1:].view(2, 8, 64)
        f(odd, p.g)


@pytest.mark.parametrize("T,D", [(300, 8192), (4000, 64)])       # alone, and in clusters
def test_bounded_waits_give_up_and_the_next_call_is_right(T, D):
    p = Problem(1, T, D, "bf16", True, seed=6)
    run = lambda: (*lib().gated_linear_recurrence_fwd(p.x, p.g, p.h0, None, p.scale),
                   *lib().gated_linear_recurrence_bwd(p.dh, p.g, p.x, p.dht, p.h0, None, p.scale))
    want, stream = run(), torch.cuda.current_stream().cuda_stream
    try:
        lib().gdn_set_spin_limit(0)
        lib().gated_linear_recurrence_fwd(p.x, p.g, p.h0, None, p.scale)
        assert lib().gdn_sync_status(stream) == 5
        lib().gated_linear_recurrence_bwd(p.dh, p.g, p.x, p.dht, p.h0, None, p.scale)
        assert lib().gdn_sync_status(stream) == 5
    finally:
        lib().gdn_set_spin_limit(-1)
    assert all(torch.equal(a, b) for a, b in zip(run(), want))
    assert lib().gdn_sync_status(stream) == 0


@pytest.mark.parametrize("D", [64 * 20, 500])
def test_packed_batches_of_several_waves(D):
    """More sequences than one wave of CTAs: they are taken longest first, equal and empty ones
    among them, by single CTAs or clusters; the results are those of each sequence alone."""
    lengths = [3, 0, 700, 700, 64, 1, 0, 1500, 129, 700, 2, 256, 31, 1500, 90, 5, 128, 127, 640, 77]
    p = Problem(0, 0, D, "bf16", True, lengths=lengths, seed=D)
    h, ht = lib().gated_linear_recurrence_fwd(p.x, p.g, p.h0, p.cu, p.scale)
    want, E, want_t, Et = reference_fwd(p)
    close("h", h, want, E, "bf16")
    close("final state", ht, want_t, Et, "fp32")
    got = lib().gated_linear_recurrence_bwd(p.dh, p.g, h, p.dht, p.h0, p.cu, p.scale)
    out, err = reference_bwd(p, h)
    for name, t in zip(("dx", "dg", "dh0", "ds"), got):
        close(name, t, out[name], err[name], "bf16" if name in ("dx", "dg") else "fp32")
    again = lib().gated_linear_recurrence_bwd(p.dh, p.g, h, p.dht, p.h0, p.cu, p.scale)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0
