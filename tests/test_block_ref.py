"""The written-out gradients of the tests' 64-bit scan against torch's differentiation of it."""
import pytest
import torch

from block_ref import scan, scan_magnitudes, spans


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 10]])
@pytest.mark.parametrize("logits,gate", [(True, True), (False, False)])
def test_the_written_out_gradients(cu, logits, gate):
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    B, T, D, S = (2, 5, 3, 4) if cu is None else (1, 10, 3, 4)
    N, n = (B if cu is None else len(cu) - 1), B * T
    v = dict(x=r(n, D), dt=r(n, D) if logits else r(n, D).abs(), a=-r(D, S).abs(), b=r(n, S), c=r(n, S), skip=r(D),
             z=r(n, D) if gate else None, dt_bias=r(D) if logits else None, h0=r(N, D, S))
    leaves = {k: t.requires_grad_() for k, t in v.items() if t is not None}
    dy, dht, seqs = r(n, D), r(N, D, S), spans(B, T, cu)
    y, states = scan(**v, seqs=seqs)
    grads = dict(zip(leaves, torch.autograd.grad([y, states], list(leaves.values()), [dy, dht])))
    with torch.no_grad():
        got = scan_magnitudes(**v, dy=dy, dht=dht, seqs=seqs, signed=True)
    torch.testing.assert_close(got["y"], y)
    torch.testing.assert_close(got["state"], states)
    for k, g in grads.items():
        torch.testing.assert_close(got["d" + k], g)
