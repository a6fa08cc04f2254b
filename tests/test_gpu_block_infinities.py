"""Infinite inputs of the state space block's operators: what the definitions give for them, and no
further than they reach."""
import pytest
import torch

from block_ref import HALF_STEP, inside
from gpu_helpers import lib
from test_gpu_ffn import ADD, gpu, make

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
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


@pytest.mark.parametrize("M", [4, 300])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_slopes_of_the_largest_projections(M, name):
    """Gates whose square fp32 does not hold: the slope is 0 or 1."""
    gdn = lib()
    p = make(M, 64, 64)
    p["gate"] = torch.tensor([-1e20, 1e20, -3e38, 3e38, -2e19, 2e19, -1e30, 1e30] * 8).expand(M, 64).contiguous().to(BF)
    out = gdn.gated_feed_forward_bwd(*gpu(p, "dy", "x", "w_gate", "w_up", "w_down", "gate", "up"), activation=name)
    dy, wd, u, x = (p[k].double() for k in ("dy", "w_down", "up", "x"))
    on = (p["gate"] > 0).double()
    dg = (dy @ wd) * u * on
    edg = 64 * ADD * (dy.abs() @ wd.abs()) * u.abs() * on
    half = HALF_STEP[BF]
    edg = edg + half * (dg.abs() + edg)
    want = dg.T @ x
    e = edg.T @ x.abs() + M * ADD * ((dg.abs() + edg).T @ x.abs())
    inside("dw_gate", out[1], want, e + half * (want.abs() + e))
