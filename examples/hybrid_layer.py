"""A recurrent layer that runs the package's operators together: the residual addition
with the RMS norm to MXFP8, the 8-bit in-projection, the gated delta rule beside the
per-channel gated linear recurrence, and the 4-bit out-projection.  Prefill, decode token by
token from the prefill's states, and a few training steps.

    python examples/hybrid_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_bwd_gb300 as gdn  # noqa: E402

K = 128          # head size of the delta rule


class HybridLayer:
    """y = W4 [recurrence(u), delta rule(q, k, v)] of the normed sum x + residual."""

    def __init__(self, width, heads, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen)
        self.width, self.heads = width, heads
        parts = [width, width] + [heads * K] * 3
        self.splits = parts
        self.norm = torch.ones(width, dtype=torch.bfloat16, device=device)
        # weights are laid out once: 8 bits into the layer, 4 out of it
        self.w_in = gdn.mx_quantize((rand(sum(parts), width) * width ** -0.5).bfloat16().to(device), "mxfp8")
        self.w_out = gdn.mx_quantize((rand(width, width + heads * K) * (2 * width) ** -0.5).bfloat16().to(device), "mxfp4")
        self.w_gate = (rand(2 * heads, width) * width ** -0.5).bfloat16().to(device)
        self.decay = (torch.rand(width, generator=gen) + 0.01).to(device)
        self.head_decay = (torch.rand(heads, generator=gen) + 0.01).to(device)

    def states(self, batch):
        return (torch.zeros(batch, self.width, device="cuda"), torch.zeros(batch, self.heads, K, K, device="cuda"))

    def _project(self, x, residual):
        normed, s, _ = gdn.add_rms_norm_fwd(x, self.norm, residual=residual, out="mxfp8")
        u, gate, q, k, v = gdn.mx_linear(normed, self.w_in).split(self.splits, -1)
        logits, beta = (gdn.mx_dequantize(normed, torch.bfloat16) @ self.w_gate.T).float().chunk(2, -1)
        return s, [t.contiguous() for t in (u, gate, q, k, v, logits, torch.sigmoid(beta))]

    def prefill(self, x, residual, states):
        """x, residual [B, T, width]: (y, their sum, new states)."""
        B, T, _ = x.shape
        s, (u, gate, q, k, v, logits, beta) = self._project(x, residual)
        h, h_state = gdn.gated_linear_recurrence_fwd(u.view(B, T, -1), gate.view(B, T, -1), states[0],
                                                     gate_scale=self.decay)
        heads = lambda t: t.view(B, T, self.heads, -1)
        o, d_state = gdn.chunk_gated_delta_rule_fwd(heads(q), heads(k), heads(v), logits.view(B, T, -1),
                                                    beta.view(B, T, -1), initial_state=states[1],
                                                    use_qk_l2norm=True, gate_scale=self.head_decay)
        y = gdn.mx_linear(torch.cat([h, o.reshape(B, T, -1)], -1), self.w_out)
        return y, s, (h_state, d_state)

    def step(self, x, residual, states):
        """One token: x, residual [B, width]; the states are updated in place."""
        s, (u, gate, q, k, v, logits, beta) = self._project(x, residual)
        h = gdn.gated_linear_recurrence_step(u, gate, states[0], gate_scale=self.decay)
        heads = lambda t: t.view(-1, self.heads, K)
        o = gdn.recurrent_step(heads(q), heads(k), heads(v), logits, beta, states[1], use_qk_l2norm=True,
                               gate_scale=self.head_decay)
        return gdn.mx_linear(torch.cat([h, o.flatten(1)], -1), self.w_out), s


def prefill_then_decode(width=512, heads=4, batch=2, prompt=200, tokens=8, seed=0):
    """The largest difference between decoding `tokens` tokens after a prefill of `prompt` and one
    prefill over all of them, relative to the largest output."""
    layer = HybridLayer(width, heads, seed)
    gen = torch.Generator().manual_seed(seed + 1)
    x, r = (torch.randn(batch, prompt + tokens, width, generator=gen).bfloat16().cuda() for _ in range(2))
    whole, _, whole_states = layer.prefill(x, r, layer.states(batch))
    y, _, states = layer.prefill(x[:, :prompt].contiguous(), r[:, :prompt].contiguous(), layer.states(batch))
    outs = [y] + [layer.step(x[:, t].contiguous(), r[:, t].contiguous(), states)[0][:, None]
                  for t in range(prompt, prompt + tokens)]
    rel = lambda a, b: float((a.float() - b.float()).abs().max() / b.float().abs().max())
    return rel(torch.cat(outs, 1), whole), max(rel(a, b) for a, b in zip(states, whole_states))


def train(steps=30, width=256, T=128, seed=0):
    """Losses of fitting norm -> recurrence to a target of the same form, by gradient descent."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen).cuda()
    x, residual, gate = rand(2, T, width), rand(2, T, width), rand(2, T, width)
    w, scale = torch.ones(width, device="cuda"), torch.full((width,), 0.5, device="cuda")

    def model(w, scale):
        y, s = gdn.add_rms_norm(x, w, residual)
        return gdn.gated_linear_recurrence(y, gate, gate_scale=scale)[0] + s

    target = model(1 + 0.3 * rand(width), torch.rand(width, generator=gen).cuda() + 0.2)
    losses = []
    for _ in range(steps):
        w, scale = w.detach().requires_grad_(), scale.detach().requires_grad_()
        loss = (model(w, scale) - target).square().mean()
        dw, ds = torch.autograd.grad(loss, (w, scale))
        with torch.no_grad():
            w, scale = w - 20 * dw, (scale - 5 * ds).clamp(min=0.01)
        losses.append(float(loss.detach()))
    return losses


if __name__ == "__main__":
    out, state = prefill_then_decode()
    print(f"prefill + decode against one prefill: outputs differ by {out:.2e}, states by {state:.2e} of their largest")
    losses = train()
    print(f"training: loss {losses[0]:.3e} -> {losses[-1]:.3e} in {len(losses)} steps")
