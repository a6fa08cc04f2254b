"""Gradients through the state space block's operators as autograd delivers and asks for them."""
import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def rand(*shape, seed=0, dtype=F):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def inputs(dtype=F, B=2, T=9, D=16, S=5):
    """Leaves of the convolution, the scan and the block."""
    conv = [rand(B, T, D, seed=1, dtype=dtype), rand(D, 4, seed=2, dtype=dtype), rand(D, seed=3, dtype=dtype),
            rand(B, 3, D, seed=4, dtype=dtype)]
    scan = [rand(B, T, D, seed=5, dtype=dtype), rand(B, T, D, seed=6, dtype=dtype), -rand(D, S, seed=7).abs(),
            rand(B, T, S, seed=8, dtype=dtype), rand(B, T, S, seed=9, dtype=dtype), rand(D, seed=10),
            rand(B, T, D, seed=11, dtype=dtype), rand(D, seed=12), rand(B, D, S, seed=13)]
    ffn = [rand(B, T, D, seed=14, dtype=BF), *(rand(24, D, seed=s, dtype=BF) for s in (15, 16)), rand(D, 24, seed=17, dtype=BF)]
    return conv, scan, ffn


def leaves(ts):
    return [t.clone().requires_grad_() for t in ts]


@pytest.mark.parametrize("dtype", [BF, F])
def test_a_loss_of_the_final_states_alone(dtype):
    conv, scan, _ = inputs(dtype)
    for op, ts, bwd, at in (
            (lib().causal_convolution, conv, lambda g, *a: lib().causal_convolution_bwd(torch.zeros_like(a[0]), *a[:3], g, a[3]), 4),
            (lib().state_space_scan, scan, lambda g, *a: lib().state_space_scan_bwd(torch.zeros_like(a[0]), *a[:8], g, a[8]), 9)):
        ls = leaves(ts)
        _, state = op(*ls, output_final_state=True)
        up = rand(*state.shape, seed=20, dtype=state.dtype)
        got = torch.autograd.grad(state, ls, up, allow_unused=True)
        for g, w in zip(got, bwd(up, *ts)[:at]):
            assert torch.equal(g, w.to(g.dtype))


def test_gradients_that_are_expanded_or_shifted():
    """A sum's gradient is one number expanded; a slice's begins on any address."""
    conv, scan, ffn = inputs(BF, D=24)
    for op, ts in ((lib().causal_convolution, conv), (lib().state_space_scan, scan), (lib().gated_feed_forward, ffn)):
        first = lambda r: r[0] if isinstance(r, tuple) else r
        ls = leaves(ts)
        y = first(op(*ls))
        want = torch.autograd.grad(y, ls, torch.ones_like(y), retain_graph=True)
        got = torch.autograd.grad(y.sum(), ls, retain_graph=True)
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        z, up = rand(3, seed=21, dtype=BF), rand(3 + y.numel(), seed=22, dtype=BF)
        assert up[3:].data_ptr() % 16
        got = torch.autograd.grad((torch.cat([z, y.flatten()]) * up).sum(), ls, retain_graph=True)
        want = torch.autograd.grad(y, ls, up[3:].view_as(y).clone())
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_some_leaves_only():
    """Whatever needs no gradient gets none, and the others' are the same."""
    conv, scan, ffn = inputs(BF)
    for op, ts in ((lib().causal_convolution, conv), (lib().state_space_scan, scan), (lib().gated_feed_forward, ffn)):
        loss = lambda r: (r[0] if isinstance(r, tuple) else r).float().square().sum()
        ls = leaves(ts)
        want = torch.autograd.grad(loss(op(*ls)), ls)
        for i, t in enumerate(ts):
            only = t.clone().requires_grad_()
            loss(op(*[only if j == i else u for j, u in enumerate(ts)])).backward()
            assert torch.equal(only.grad, want[i]) and not any(u.requires_grad for u in ts)


def test_second_derivatives_are_refused():
    conv, scan, ffn = inputs()
    for op, ts in ((lib().causal_convolution, conv), (lib().state_space_scan, scan), (lib().gated_feed_forward, ffn)):
        ls = leaves(ts)
        y = op(*ls)
        y = y[0] if isinstance(y, tuple) else y
        (d,) = torch.autograd.grad(y.float().square().sum() + ls[0].float().pow(3).sum(), ls[0], create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            d.float().sum().backward()


def test_the_convolution_in_front_of_the_delta_rule():
    """q, k and v through a short convolution each, as one of all channels, then the delta rule: its gradients
    come back through the convolution's backward pass, and a prompt's last token is a step of both."""
    B, T, H, K = 2, 70, 2, 64
    D = 3 * H * K
    x, w = rand(B, T, D, seed=1, dtype=BF).requires_grad_(), (rand(D, 4, seed=2, dtype=BF) * 0.5).requires_grad_()
    g, beta = -rand(B, T, H, seed=3).abs() * 0.1, torch.sigmoid(rand(B, T, H, seed=4))

    def split(y):
        return [t.reshape(*t.shape[:-1], H, K).contiguous() for t in y.split(H * K, -1)]

    def rule(y, g, beta):
        return lib().chunk_gated_delta_rule(*split(y), g, beta, use_qk_l2norm=True, output_final_state=True)

    y, conv = lib().causal_convolution(x, w, output_final_state=True)
    o, state = rule(y, g, beta)
    state = state.detach()
    do = rand(*o.shape, seed=5, dtype=o.dtype)
    dx, dw = torch.autograd.grad(o, (x, w), do)
    leaf = y.detach().requires_grad_()
    (dy,) = torch.autograd.grad(rule(leaf, g, beta)[0], leaf, do)
    want = lib().causal_convolution_bwd(dy, x.detach(), w.detach())
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1].to(BF))
    # the prompt but for its last token, and that as a step
    with torch.no_grad():
        cut = lambda t: t[:, :-1].contiguous()
        y1, conv1 = lib().causal_convolution(cut(x), w, output_final_state=True)
        assert torch.equal(y1, cut(y))
        _, state1 = rule(y1, cut(g), cut(beta))
        yt = lib().causal_convolution_step(x[:, -1].contiguous(), w, conv1)
        assert torch.equal(yt, y[:, -1]) and torch.equal(conv1, conv)
        q, k, v = split(yt)
        ot = lib().recurrent_step(q, k, v, g[:, -1].contiguous(), beta[:, -1].contiguous(), state1, use_qk_l2norm=True)
    # the delta rule's own tolerance for bf16 tensors
    assert float((ot.float() - o.detach()[:, -1].float()).abs().max()) <= 2e-2 and float((state1 - state).abs().max()) <= 2e-2
