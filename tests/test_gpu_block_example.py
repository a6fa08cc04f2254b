"""The state space block: its operators one after another, as a model runs them.

Decode and prefill take the same tokens through the same formulas.  Between them lie torch's bf16
products, whose order of summation may differ with their size (2^-8 of a result now and then), so that
a few roundings of 2^-8 travel through the block: each of its seven stages passes a relative change on
by its norm, of the order of one here, and the largest output is some four times the usual one.  5% of
the largest output, and 2% of the largest state, is room for all of them at once."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "state_space_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("state_space_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("width,hidden,batch,prompt,tokens", [(256, 512, 3, 100, 6), (128, 344, 1, 1, 5), (512, 1024, 2, 333, 3)])
def test_decode_continues_the_prefill(example, width, hidden, batch, prompt, tokens):
    y, conv, scan = example.prefill_then_decode(width, hidden, batch, prompt, tokens, seed=prompt)
    assert y < 5e-2 and conv < 2e-2 and scan < 2e-2


def test_packed_sequences_are_their_own(example):
    assert example.packed_against_rows([5, 1, 0, 64, 30, 3]) < 5e-2


def plain(block, x, residual):
    """The block in 64 bits, from its formulas."""
    p = block.p
    norm = lambda s, w: s * torch.rsqrt(s.square().mean(-1, keepdim=True) + 1e-6) * w
    s = x + residual
    u, z = (norm(s, p["norm1"]) @ p["w_in"].T).split(block.inner, -1)
    W = p["conv"].shape[1]
    padded = torch.nn.functional.pad(u, (0, 0, W - 1, 0))
    u = p["conv_bias"] + sum(p["conv"][:, k] * padded[:, k:k + u.shape[1]] for k in range(W))
    u = torch.nn.functional.silu(u)
    dt, b, c = (u @ p["w_x"].T).split([p["w_dt"].shape[1], p["a"].shape[1], p["a"].shape[1]], -1)
    delta = torch.nn.functional.softplus(dt @ p["w_dt"].T + p["dt_bias"])
    h, ys = torch.zeros(*u[:, 0].shape, p["a"].shape[1], dtype=u.dtype, device=u.device), []
    for t in range(u.shape[1]):
        h = torch.exp(delta[:, t, :, None] * p["a"]) * h + (delta[:, t] * u[:, t])[..., None] * b[:, t, None]
        ys.append((h * c[:, t, None]).sum(-1))
    y = (torch.stack(ys, 1) + p["skip"] * u) * torch.nn.functional.silu(z)
    s = s + y @ p["w_out"].T
    n = norm(s, p["norm2"])
    return (torch.nn.functional.silu(n @ p["w_gate"].T) * (n @ p["w_up"].T)) @ p["w_down"].T, s


def test_gradients_of_a_training_step(example):
    """Against the 64-bit block's: some ten tensors on the way are rounded to bf16, forward and back, by
    2^-8 / sqrt(3) of themselves on average, independently: 2^-8 (20 / 3)^(1/2) = 1% of a gradient's norm.
    Three times that for what the block amplifies."""
    loss, grads = example.training_step()
    block = example.StateSpaceBlock(128, 256, 0)
    block.p = {k: t.double().requires_grad_() for k, t in block.p.items()}
    x, r = (t.double().requires_grad_() for t in example.inputs(2, 70, 128, 1))
    target, _ = example.inputs(2, 70, 128, 2)
    y, s = plain(block, x, r)
    want_loss = ((y + s) - target.double()).square().mean()
    leaves = {"x": x, "residual": r, **block.p}
    want = dict(zip(leaves, torch.autograd.grad(want_loss, list(leaves.values()))))
    assert abs(loss - float(want_loss.detach())) <= 0.01 * float(want_loss.detach())
    for k, g in grads.items():
        assert g.dtype == (torch.float32 if k in ("a", "skip", "dt_bias") else torch.bfloat16), k
        off = float((g.double() - want[k]).norm() / want[k].norm())
        assert off <= 0.03, (k, off)
