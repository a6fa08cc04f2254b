"""The scan's exponentials, logarithms and logistic functions one by one: what fp32 tensors are promised,
and which way the decays lean."""
import math

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


def as_step(p):
    return {k: t[:, 0].contiguous() if t.dim() == 3 else t for k, t in p.items()}


def state_of(p, start, step):
    """The state after the token, [D], from `start`."""
    h0 = torch.full((1, D, 1), float(start), device="cuda")
    if step:
        lib().state_space_step(state=h0, **as_step(p))
        return h0.view(-1)
    return lib().state_space_scan_fwd(initial_state=h0, **p)[1].view(-1)


LOGITS = torch.cat([torch.linspace(-80, 20, D - 1024), torch.linspace(-2, 2, 1024)]).view(1, 1, D)


@pytest.mark.parametrize("step", [False, True])
def test_softplus_of_fp32(step):
    """From no state the new state is delta x b = delta: log1p(e^v), whose argument is off by 2 U."""
    want = torch.nn.functional.softplus(LOGITS.double(), threshold=100).view(-1)
    inside("delta", state_of(one_token(dt=LOGITS, dt_bias=torch.zeros(D)), 0, step), want, 5 * U * want)


@pytest.mark.parametrize("step", [False, True])
def test_gate_of_fp32(step):
    """Of a state that stays zero y is skip x silu(z) = z / (1 + e^-z): 2 U and three roundings."""
    p = one_token(z=LOGITS, skip=torch.ones(D), b=torch.zeros(1, 1, 1))
    if step:
        y = lib().state_space_step(state=torch.zeros(1, D, 1, device="cuda"), **as_step(p))
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
    inside("dz", dz.view(-1), want, s * rest + (4 * U + U) * want.abs())


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("dtype", [BF, F])
def test_a_decay(dtype, step):
    """A state of 1 after one token: the hardware's exponential is off by 2^-22, its argument by three
    roundings (log2 e, its product with a, that with the step) and the 1.2e-8 that bf16 tensors' have added.
    For fp32 and |delta a| < 1/32 ln 2 the polynomial: its last rounding, 1.1e-7 |y|, and the argument's."""
    dt = torch.cat([torch.logspace(-5, math.log10(80), D - 2048), torch.linspace(0, 0.0216, 2048)]).view(1, 1, D).to(dtype)
    p = {k: t.to(dtype) if k in "xbc" else t for k, t in one_token(x=torch.zeros(1, 1, D), dt=dt).items()}
    v = dt.double().view(-1)
    want = torch.exp(-v)
    room = 2.0 ** -22 + 3 * U * v + (1.2e-8 if dtype == BF else 0)
    if dtype == F:
        room = torch.where(v < 0.0216, U + 1.1e-7 * v / math.log(2) + 3 * U * v, room)
    inside("state", state_of(p, 1, step), want, room * want)


def lean(dt, dtype):
    """What a decay is too small (below 0) or too large by, on average, for steps dt [128, D] times a = -1.  The
    state is a product of 128 of them, short enough to be walked whole (where a sequence is cut, a part's decay
    is one exponential), in which roundings to either side average out over the channels: 1024 x 1024 of
    U / sqrt(3) each, 3e-11."""
    T = dt.shape[0]
    dt = dt.to(dtype)[None]
    none, one = torch.zeros(1, T, D, dtype=dtype), torch.zeros(1, T, 1, dtype=dtype)
    n = lib()._abi_layer.ENTRIES["gdn_ssm_fwd"]
    assert n.workspace_size(n.pack(*[0] * 10, 1, T, D, 1, 1, 1 if dtype == BF else 0, 0, 0)) == 256      # whole
    _, ht = lib().state_space_scan_fwd(none.cuda(), dt.cuda(), -torch.ones(D, 1).cuda(), one.cuda(), one.cuda(),
                                       initial_state=torch.ones(1, D, 1).cuda())
    off = torch.log(ht[0, :, 0].cpu().double()) + dt.double().sum(1)[0]
    return float(off.mean()) / T


def between(lo, hi):
    return lo + (hi - lo) * torch.rand(128, D, generator=torch.Generator().manual_seed(3))


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("lo,hi", [(1e-4, 5e-4), (5e-4, 4e-3), (4e-3, 2e-2), (2e-2, 4e-2)])
def test_decays_hardly_lean(dtype, lo, hi):
    """The hardware's exponential is low by 0.5e-8 to 3.3e-8, as its argument goes; of bf16 tensors, whose
    arguments have ln 2 1.73e-8 = 1.2e-8 added, 2.1e-8 is left at most."""
    assert abs(lean(between(lo, hi), dtype)) <= (2.1e-8 if dtype == BF else 3.3e-8)


def test_decays_lean_neither_way():
    """Over the steps that a layer begins with, by their logarithm: the exponential's lean is 1.8e-8 there (its
    mean over the same steps, measured by itself), with the constant that bf16 tensors have 0.6e-8: less than the
    constant itself, which a sum without it is not.  And of fp32 tensors' polynomial 1.1e-7 of the argument."""
    steps = torch.exp(between(math.log(1e-3), math.log(0.1)))
    assert abs(lean(steps, BF)) <= 1.2e-8
    slow = between(5e-4, 2e-2)
    assert abs(lean(slow, F)) <= 1.1e-7 * float(slow.mean()) / math.log(2) + 1e-10
