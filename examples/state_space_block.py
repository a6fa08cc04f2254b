"""A block of a state space language model from the package's operators: residual + RMS norm, a
projection, the short causal convolution, the selective state space scan with its gate, and behind a
second norm the gated feed-forward block.  Prefill, decode token by token from the prefill's states,
and the gradients of a training step.

    python examples/state_space_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_bwd_gb300 as gdn  # noqa: E402

STATES, TAPS, RANK = 16, 4, 32       # of the scan, of the convolution, of the steps' projection


class StateSpaceBlock:
    """y = FFN(norm(s)) with s = x + residual + mixer(norm(x + residual))."""

    def __init__(self, width, hidden, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen)
        bf = lambda t: t.bfloat16().to(device)
        self.width, self.inner = width, 2 * width
        self.p = dict(
            norm1=bf(torch.ones(width)), norm2=bf(torch.ones(width)),
            w_in=bf(rand(2 * self.inner, width) * width ** -0.5),
            conv=bf(rand(self.inner, TAPS) * TAPS ** -0.5), conv_bias=bf(0.1 * rand(self.inner)),
            w_x=bf(rand(RANK + 2 * STATES, self.inner) * self.inner ** -0.5),
            w_dt=bf(rand(self.inner, RANK) * RANK ** -0.5), dt_bias=(torch.rand(self.inner, generator=gen) * 4 - 6).to(device),
            a=-torch.arange(1.0, STATES + 1).expand(self.inner, STATES).contiguous().to(device),
            skip=torch.ones(self.inner, device=device), w_out=bf(rand(width, self.inner) * self.inner ** -0.5),
            w_gate=bf(rand(hidden, width) * width ** -0.5), w_up=bf(rand(hidden, width) * width ** -0.5),
            w_down=bf(rand(width, hidden) * hidden ** -0.5))

    def states(self, batch):
        return (torch.zeros(batch, TAPS - 1, self.inner, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(batch, self.inner, STATES, device="cuda"))

    def parameters_of_the_scan(self, u):
        dt, b, c = (u @ self.p["w_x"].T).split([RANK, STATES, STATES], -1)
        return (dt @ self.p["w_dt"].T).contiguous(), b.contiguous(), c.contiguous()

    def __call__(self, x, residual, states=None, cu_seqlens=None):
        """x, residual [B, T, width] (with cu_seqlens one row of packed sequences): (y, sum, new states);
        differentiable in everything."""
        p = self.p
        conv0, scan0 = states if states is not None else (None, None)
        normed, s = gdn.add_rms_norm(x, p["norm1"], residual)
        u, z = (normed @ p["w_in"].T).split(self.inner, -1)
        u, conv1 = gdn.causal_convolution(u.contiguous(), p["conv"], p["conv_bias"], conv0, cu_seqlens,
                                          output_final_state=True)
        dt, b, c = self.parameters_of_the_scan(u)
        y, scan1 = gdn.state_space_scan(u, dt, p["a"], b, c, p["skip"], z.contiguous(), p["dt_bias"], scan0, cu_seqlens,
                                        output_final_state=True)
        normed, s = gdn.add_rms_norm(y @ p["w_out"].T, p["norm2"], s)
        return gdn.gated_feed_forward(normed, p["w_gate"], p["w_up"], p["w_down"]), s, (conv1, scan1)

    def step(self, x, residual, states):
        """One token: x, residual [B, width]; the states are updated in place."""
        p = self.p
        normed, s, _ = gdn.add_rms_norm_fwd(x, p["norm1"], residual=residual)
        u, z = (normed @ p["w_in"].T).split(self.inner, -1)
        u = gdn.causal_convolution_step(u.contiguous(), p["conv"], states[0], p["conv_bias"])
        dt, b, c = self.parameters_of_the_scan(u)
        y = gdn.state_space_step(u, dt, p["a"], b, c, states[1], p["skip"], z.contiguous(), p["dt_bias"])
        normed, s, _ = gdn.add_rms_norm_fwd(y @ p["w_out"].T, p["norm2"], residual=s)
        return gdn.gated_feed_forward_fwd(normed, p["w_gate"], p["w_up"], p["w_down"])[0], s


def inputs(batch, tokens, width, seed):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(batch, tokens, width, generator=gen).bfloat16().cuda() for _ in range(2)]


def difference(a, b):
    """The largest difference, relative to the largest value."""
    return float((a.float() - b.float()).abs().max() / b.float().abs().max())


@torch.no_grad()
def prefill_then_decode(width=256, hidden=512, batch=3, prompt=100, tokens=6, seed=0):
    """How far decoding `tokens` tokens after a prefill of `prompt` is from one prefill over all of them:
    of the outputs, of the convolution's states, of the scan's."""
    block = StateSpaceBlock(width, hidden, seed)
    x, r = inputs(batch, prompt + tokens, width, seed + 1)
    whole, _, whole_states = block(x, r, block.states(batch))
    y, _, states = block(x[:, :prompt].contiguous(), r[:, :prompt].contiguous(), block.states(batch))
    outs = [y] + [block.step(x[:, t].clone(), r[:, t].clone(), states)[0][:, None] for t in range(prompt, prompt + tokens)]
    return difference(torch.cat(outs, 1), whole), *(difference(a, b) for a, b in zip(states, whole_states))


@torch.no_grad()
def packed_against_rows(lengths, width=256, hidden=512, seed=0):
    """How far one packed batch of sequences is from each of them by itself."""
    block = StateSpaceBlock(width, hidden, seed)
    ends = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    x, r = inputs(1, ends[-1], width, seed + 1)
    y, _, _ = block(x, r, cu_seqlens=torch.tensor(ends, dtype=torch.int32, device="cuda"))
    rows = [block(x[:, a:b].clone(), r[:, a:b].clone())[0] for a, b in zip(ends, ends[1:]) if b > a]
    return difference(y, torch.cat(rows, 1))


def training_step(width=128, hidden=256, batch=2, tokens=70, seed=0):
    """The loss of a random target and its gradients: (loss, {name: gradient}) with the inputs' first."""
    block = StateSpaceBlock(width, hidden, seed)
    x, r = (t.requires_grad_() for t in inputs(batch, tokens, width, seed + 1))
    leaves = {"x": x, "residual": r, **{k: t.requires_grad_() for k, t in block.p.items()}}
    target, _ = inputs(batch, tokens, width, seed + 2)
    y, s, _ = block(x, r)
    loss = ((y + s).float() - target.float()).square().mean()
    return float(loss.detach()), dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))


if __name__ == "__main__":
    y, conv, scan = prefill_then_decode()
    print(f"prefill + decode against one prefill: outputs {y:.2e}, convolution's states {conv:.2e}, scan's {scan:.2e}")
    print(f"packed sequences against single ones: {packed_against_rows([5, 1, 64, 30]):.2e}")
    loss, grads = training_step()
    print(f"training step: loss {loss:.4f}, largest gradients " +
          ", ".join(f"{k} {float(g.abs().max()):.1e}" for k, g in grads.items()))
