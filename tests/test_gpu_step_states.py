"""Where a step's new states go: over the old ones, right behind or before them, nowhere half over them."""
import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def steps(dtype, N=4, D=24, S=16):
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen)
    c = lambda *s: r(*s).to(dtype).cuda()
    x, w, g, dt, b, cc = c(N, D), c(D, 4), c(N, D), c(N, D).abs(), c(N, S), c(N, S)
    a = -r(D, S).abs().cuda()
    return [((N, 3, D), dtype, lambda st, out: lib().causal_convolution_step(x, w, st, out_state=out)),
            ((N, D, S), F, lambda st, out: lib().state_space_step(x, dt, a, b, cc, st, out_state=out)),
            ((N, D), F, lambda st, out: lib().gated_linear_recurrence_step(x, -g.abs(), st, out_state=out))]


@pytest.mark.parametrize("dtype", [BF, F])
def test_where_new_states_go(dtype):
    for shape, kind, step in steps(dtype):
        N = shape[0]
        first = torch.randn(shape, generator=torch.Generator().manual_seed(1)).to(kind).cuda()
        apart = torch.empty_like(first)
        y = step(first, apart)
        own = first.clone()
        assert torch.equal(step(own, None), y) and torch.equal(own, apart)
        pool = torch.zeros(2 * N, *shape[1:], dtype=kind, device="cuda")
        for old, new in ((pool[:N], pool[N:]), (pool[N:], pool[:N])):
            old.copy_(first)
            assert torch.equal(step(old, new), y) and torch.equal(new, apart) and torch.equal(old, first)
        for old, new in ((pool[:N], pool[1:N + 1]), (pool[1:N + 1], pool[:N])):
            with pytest.raises(lib().GdnError, match="overlaps"):
                step(old, new)
