"""Gate logits of slow channels: steady logits of -4 to -20 under gate scales up to 16, thousands of
tokens long, so that a channel's state and d(gate_scale) rest on the small softplus(g) ~ e^g.

Tolerances, relative to softplus itself.  u = 2^-24.  e^g from a rounded product and an exponential:
(2 |g| + 4) u; log(1 + e^g) from it, 12 u more; so softplus is off by r = (2 |g| + 16) u of itself.
The log decay l = -a softplus(g) adds two roundings, the decay e^l one of its result (half an ulp below
1, which its own error of 6e-10 leaves), and a step of the walk one: e^l is off by |l| (r + 2 u) + 2 u of
itself, and the states follow E_t = a_t E_{t-1} + that times m_t with m_t = a_t m_{t-1} + |x_t|.  A tile
of 32 tokens or more ends in four further products: 4 u m at each, of which there are T / 32.
d(gate_scale) is a sum of -softplus(g) dl: each term carries r and its dl's error, and the sums in fp32
64 u of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
LOGITS = np.array([-4, -6, -8, -10, -12, -13, -14, -15, -16, -16.5, -17, -18, -20, -3, -5, -11])
SCALES = np.array([16.0, 8.0, 1.0, 4.0])


class Slow:
    """Logits of one value per channel (exact in bf16), every pair of LOGITS and SCALES among them."""

    def __init__(self, B, T, D, dtype, seed):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.rand(*s, generator=gen) + 0.5
        k = np.arange(D)
        self.logit, self.a = LOGITS[k % 16], SCALES[k // 16 % 4]
        dt = DT[dtype]
        self.x, self.dh = rand(B, T, D).to(dt).cuda(), rand(B, T, D).to(dt).cuda()
        self.g = torch.tensor(self.logit).to(dt).cuda().expand(B, T, D).contiguous()
        assert np.array_equal(self.g[0, 0].double().cpu().numpy(), self.logit) if T else True
        self.scale = torch.tensor(self.a, dtype=torch.float32).cuda()
        self.h0, self.dht = rand(B, D).cuda(), rand(B, D).cuda()
        self.sp = np.log1p(np.exp(self.logit))
        self.r = (2 * np.abs(self.logit) + 16) * U
        self.decay = np.exp(-self.a * self.sp)
        self.c = self.a * self.sp * (self.r + 2 * U) + 2 * U + 4 * U / 32


def np64(t):
    return t.double().cpu().numpy()


def within(name, got, want, tol):
    bad = ~(np.abs(np64(got) - want) <= tol)
    assert not bad.any(), (name, int(bad.sum()), float((np.abs(np64(got) - want) / tol).max()))


# few channels (cut into parts), clusters, single CTAs, and rows that TMA does not take
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,D", [(1, 8192, 64), (2, 6000, 512), (3, 4096, 8192), (1, 5000, 67)])
def test_slow_channels_keep_their_decay(B, T, D, dtype):
    p = Slow(B, T, D, dtype, seed=T + D)
    h, ht = lib().gated_linear_recurrence_fwd(p.x, p.g, p.h0, None, p.scale)
    x, now = np64(p.x), np64(p.h0)
    E = np.zeros_like(now)
    for t in range(T):
        now = p.decay * now + x[:, t]
        E = p.decay * E + p.c * now          # everything is positive: m is the state
    within("final state", ht, now, E + 8 * U * now)

    # from states that stay near 1, so that no stored state's rounding enters
    saved = torch.ones_like(p.x)
    _, dg, dh0, ds = lib().gated_linear_recurrence_bwd(p.dh, p.g, saved, p.dht, p.h0, None, p.scale)
    dh, c = np64(p.dh), np64(p.dht)
    e = np.zeros_like(c)
    want, tol = np.zeros(D), np.zeros(D)
    for t in range(T - 1, -1, -1):
        c, e = p.decay * (dh[:, t] + c), p.decay * e + p.c * p.decay * (dh[:, t] + c)
        dl = c * (np64(p.h0) if t == 0 else 1.0)
        want -= (p.sp * dl).sum(0)
        tol += (p.sp * ((e / c + p.r + 4 * U) * dl)).sum(0)
    within("dh0", dh0, c, e + 8 * U * c)
    within("d(gate_scale)", ds, want, tol + 64 * U * np.abs(want))
    # dg of the first token: -a sigmoid(g) dl
    sig = 1 / (1 + np.exp(-p.logit))
    first = -p.a * sig * c * np64(p.h0)
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    within("dg", dg[:, 0], first, np.abs(first) * (half + e / c + p.r + 16 * U))
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decoding_goes_on_with_the_prefills_decay(dtype):
    """A prefill of 4000 tokens, then 3000 single ones, against one prefill of all 7000: the fp32
    states agree within both sides' bounds."""
    T, more = 4000, 3000
    p = Slow(2, T + more, 256, dtype, seed=3)
    cut = lambda t, lo, hi: t[:, lo:hi].contiguous()
    _, state = lib().gated_linear_recurrence_fwd(cut(p.x, 0, T), cut(p.g, 0, T), p.h0, None, p.scale)
    for t in range(T, T + more):
        lib().gated_linear_recurrence_step(p.x[:, t].contiguous(), p.g[:, t].contiguous(), state, p.scale)
    _, whole = lib().gated_linear_recurrence_fwd(p.x, p.g, p.h0, None, p.scale)
    x, now = np64(p.x), np64(p.h0)
    E = np.zeros_like(now)
    for t in range(T + more):
        now = p.decay * now + x[:, t]
        E = p.decay * E + p.c * now
    within("prefill and steps", state, now, E + 8 * U * now)
    within("one prefill", whole, now, E + 8 * U * now)
