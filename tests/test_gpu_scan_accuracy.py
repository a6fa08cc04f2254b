"""The scan's exponentials, logarithms and logistic functions one by one: what fp32 tensors are promised,
and which way the decays lean."""
import pytest
import torch

from block_ref import inside, silu_slope
from gpu_helpers import lib

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
U = 2.0 ** -24                       # a rounding; CUDA's expf and log1pf are off by one place, 2 U, at most
D = 8192


def one_token(**kw):
    """A token of D channels with one state whose coefficients are 1, as [1, 1, D] tensors."""
    row, one = torch.zeros(1, 1, D), torch.ones(1, 1, 1)
    p = dict(x=torch.ones(1, 1, D), dt=row, a=torch.full((D, 1), -1.0), b=one, c=one)
    p.update(kw)
    return {k: None if t is None else t.cuda() for k, t in p.items()}


LOGITS = torch.cat([torch.linspace(-80, 20, D - 1024), torch.linspace(-2, 2, 1024)]).view(1, 1, D)


@pytest.mark.parametrize("step", [False, True])
def test_softplus_of_fp32(step):
    """From no state the new state is delta x b = delta: log1p(e^v), whose argument is off by 2 U."""
    p = one_token(dt=LOGITS, dt_bias=torch.zeros(D))
    if step:
        state = torch.zeros(1, D, 1, device="cuda")
        lib().state_space_step(state=state, **{k: t[:, 0].contiguous() if t.dim() == 3 else t for k, t in p.items()})
    else:
        _, state = lib().state_space_scan_fwd(**p)
    want = torch.nn.functional.softplus(LOGITS.double(), threshold=100)[0, 0]
    inside("delta", state[0, :, 0], want, 5 * U * want)


@pytest.mark.parametrize("step", [False, True])
def test_gate_of_fp32(step):
    """Of a state that stays zero y is skip x silu(z) = z / (1 + e^-z): 2 U and three roundings."""
    p = one_token(z=LOGITS, skip=torch.ones(D), b=torch.zeros(1, 1, 1))
    if step:
        y = lib().state_space_step(state=torch.zeros(1, D, 1, device="cuda"),
                                   **{k: t[:, 0].contiguous() if t.dim() == 3 else t for k, t in p.items()})
    else:
        y = lib().state_space_scan_fwd(**p)[0]
    z = LOGITS.double().view(-1)
    want = z * torch.sigmoid(z)
    inside("y", y.view(-1), want, 5 * U * want.abs())


def test_slopes_of_fp32():
    """With dy, x, b and c of 1: ddelta is 1, ddt the logistic function of the logit; and of the gate alone dz
    is silu's slope s (1 + z (1 - s))."""
    v = LOGITS.double().view(-1)
    s = torch.sigmoid(v)
    dy = torch.ones(1, 1, D).cuda()
    ddt = lib().state_space_scan_bwd(dy, **one_token(dt=LOGITS, dt_bias=torch.zeros(D)))[1]
    inside("ddt", ddt.view(-1), s, 4 * U * s)
    dz = lib().state_space_scan_bwd(dy, **one_token(z=LOGITS, skip=torch.ones(D), b=torch.zeros(1, 1, 1)))[6]
    es = 4 * U * s                    # of s; then 1 - s, its product, the sum and the last product
    want, rest = silu_slope(v), v.abs() * (es + U * (1 - s)) + 2 * U * (1 + v.abs() * (1 - s))
    inside("dz", dz.view(-1), want, s * rest + (es / s + U) * want.abs())


def lean(dtype, lo, hi):
    """What one decay is too small or too large by, on average, over steps of lo .. hi times a = -1: the
    state is a product of T of them, whose roundings to either side average out."""
    T, channels = 2048, 2048
    gen = torch.Generator().manual_seed(3)
    dt = (lo + (hi - lo) * torch.rand(1, T, channels, generator=gen)).to(dtype)
    none, one = torch.zeros(1, T, channels, dtype=dtype), torch.zeros(1, T, 1, dtype=dtype)
    _, ht = lib().state_space_scan_fwd(none.cuda(), dt.cuda(), -torch.ones(channels, 1).cuda(), one.cuda(), one.cuda(),
                                       initial_state=torch.ones(1, channels, 1).cuda())
    exact = -dt.double().sum(1)[0]
    return float((torch.log(ht[0, :, 0].cpu().double()) - exact).mean() / T)
