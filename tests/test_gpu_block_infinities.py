"""Infinite inputs of the state space block's operators: what the definitions give for them, and no
further than they reach."""
import pytest
import torch

from gpu_helpers import lib
from test_gpu_ffn import gpu, make

pytestmark = pytest.mark.gpu

INF = float("inf")


# ------------------------------------------------------------------ feed-forward
@pytest.mark.parametrize("M", [3, 64, 65, 300])
def test_a_feature_that_overflows(M):
    """Feature 5 is 2^141 of token 1, and of token 2 3.402e38, which fp32 holds and bf16 rounds to infinity:
    however many tokens there are, the result is infinite, with the signs of its column of w_down."""
    gdn = lib()
    p = make(M, 72, 136)
    x, wg, wu, wd = gpu(p, "x", "w_gate", "w_up", "w_down")
    wg[:, 0], wu[:, 0] = 0, 0
    wd[:, 5] = torch.where(wd[:, 5] < 0, -0.5, 0.5)
    wg[5], wu[5] = 0, 0
    wg[5, 0], wu[5, 0] = 1, 2
    x[:, 0] = 0
    without = gdn.gated_feed_forward_fwd(x, wg, wu, wd)[0]
    x[1, 0], x[2, 0] = 2.0 ** 70, 181 / 128 * 2.0 ** 63
    y = gdn.gated_feed_forward_fwd(x, wg, wu, wd)[0]
    assert torch.isfinite(without).all()
    for t in (1, 2):
        assert torch.equal(y[t].float(), wd[:, 5].float() * INF)
    keep = torch.tensor([t for t in range(M) if t not in (1, 2)])
    assert torch.equal(y[keep], without[keep])
