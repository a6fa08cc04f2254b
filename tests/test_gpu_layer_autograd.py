"""Gradients through the layer operators as autograd delivers and asks for them."""
import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu


def rand(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lead", [1, 3])
def test_gradients_may_arrive_on_any_address(lead, dtype):
    """torch.cat along the first axis hands back slices of its gradient: contiguous, but on no
    16-byte boundary where a row's bytes are no multiple of it."""
    D = 101
    x, w, g = rand(6, D, seed=1, dtype=dtype), rand(D, seed=2, dtype=dtype), rand(1, 6, D, seed=3, dtype=dtype)
    z, up = rand(lead, D, seed=4, dtype=dtype), rand(lead + 6, D, seed=5, dtype=dtype)
    zt, upt = rand(lead, D, seed=6), rand(lead + 1, D, seed=7)
    assert up[lead:].data_ptr() % 16

    def grads(join):
        a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
        y, s = lib().add_rms_norm(a, b, x)
        h, ht = lib().gated_linear_recurrence(a[None], g, output_final_state=True)
        return torch.autograd.grad(join(y, s, h[0], ht), (a, b))

    whole = lambda t, rest: torch.cat([rest, t], 0)
    got = grads(lambda y, s, h, ht: sum((whole(t, z) * up).sum() for t in (y, s, h)) + (whole(ht, zt) * upt).sum())
    aligned, aligned_t = up[lead:].clone(), upt[lead:].clone()
    want = grads(lambda y, s, h, ht: sum((t * aligned).sum() for t in (y, s, h)) + (ht * aligned_t).sum())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("lead", [(8,), (2, 4)])
def test_a_loss_through_a_microscaled_product_is_refused(lead):
    """The product has no backward pass: a gradient that reaches it raises instead of ending there
    without a word.  Calls that ask for none are what they were."""
    x, w = rand(*lead, 64, seed=1, dtype=torch.bfloat16), lib().mx_quantize(rand(32, 64, seed=2), "mxfp8")
    want = lib().mx_linear(x, w)
    assert not want.requires_grad
    y = x.clone().requires_grad_()
    with torch.no_grad():
        out = lib().mx_linear(y, w)
    assert torch.equal(out, want) and not out.requires_grad
    out = lib().mx_linear(y, w, torch.float32)
    assert torch.equal(out.detach(), lib().mx_linear(x, w, torch.float32))
    with pytest.raises(RuntimeError, match="no backward"):
        out.sum().backward()


def test_second_derivatives_are_refused():
    """The backward passes are not differentiable themselves: backward() through them raises, also
    where another path from the input has a second derivative."""
    x, w = rand(4, 64, seed=1).requires_grad_(), rand(64, seed=2)
    g = rand(1, 4, 64, seed=3)
    for f in (lambda: lib().add_rms_norm(x, w), lambda: lib().gated_linear_recurrence(x[None], g)[0]):
        (d,) = torch.autograd.grad(f().square().sum() + x.pow(3).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            d.sum().backward()
