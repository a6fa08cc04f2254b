"""The state space block's operators where offsets pass 32 bits: the last tokens of a long call against
the same tokens by themselves."""
import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
T, D, LAST = 540_000, 4096, 200                  # 2.2e9 elements, 4.4 GB


def test_convolution_past_32_bits():
    x, w = torch.randn(1, T, D, device="cuda", dtype=BF), torch.randn(D, 4, device="cuda", dtype=BF)
    y, ht = lib().causal_convolution_fwd(x, w)
    tail = x[:, -LAST:].clone()
    before = x[:, -LAST - 3:-LAST].clone()
    want, _ = lib().causal_convolution_fwd(tail, w, initial_state=before)
    assert torch.equal(y[:, -LAST:], want) and torch.equal(ht, x[:, -3:])
    # the gradient of the last tokens: those of the others are zeros
    dy = torch.zeros_like(x)
    dy[:, -LAST:] = y[:, -LAST:]
    dx, dw, _, _ = lib().causal_convolution_bwd(dy, x, w)
    some, dw2, _, dh0 = lib().causal_convolution_bwd(want, tail, w, initial_state=before)
    assert torch.equal(dx[:, -LAST:], some) and torch.equal(dx[:, -LAST - 3:-LAST], dh0)
    assert not dx[:, :1000].any()
    # two orders of a sum of 200 terms, 200 2^-24 of their magnitudes, which are below 20 each
    assert float((dw - dw2).abs().max()) <= 200 * 200 * 20 * 2.0 ** -24


def test_scan_past_32_bits():
    """Steps of 1 and a = -5: after 40 tokens nothing is left of a state (e^-200)."""
    S = 2
    x = torch.randn(1, T, D, device="cuda", dtype=BF)
    dt = torch.ones(1, T, D, device="cuda", dtype=BF)
    a = torch.full((D, S), -5.0, device="cuda")
    b, c = (torch.randn(1, T, S, device="cuda", dtype=BF) for _ in range(2))
    y, ht = lib().state_space_scan_fwd(x, dt, a, b, c)
    cut = lambda t: t[:, -LAST:].clone()
    want, ht2 = lib().state_space_scan_fwd(cut(x), cut(dt), a, cut(b), cut(c))
    # a sum over two states and some of the last tokens, each by 2^-20, and two roundings
    off = (y[:, -100:].float() - want[:, -100:].float()).abs()
    assert bool((off <= 2.0 ** -7 * want[:, -100:].float().abs() + 1e-4).all())
    assert bool(((ht - ht2).abs() <= 1e-5 * (1 + ht2.abs())).all())
    dy = torch.zeros_like(x)
    dy[:, -100:] = y[:, -100:]
    del y
    dx = lib().state_space_scan_bwd(dy, x, dt, a, b, c)[0]
    some = lib().state_space_scan_bwd(cut(dy), cut(x), cut(dt), a, cut(b), cut(c))[0]
    off = (dx[:, -100:].float() - some[:, -100:].float()).abs()
    assert bool((off <= 2.0 ** -7 * some[:, -100:].float().abs() + 1e-3).all())
    assert not dx[:, :1000].any()


def test_feed_forward_past_32_bits():
    M, K, H = 262_500, 64, 8200                  # 2.15e9 elements in the block
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen, dtype=BF)
    x, dy = r(M, K), r(M, K)
    wg, wu, wd = r(H, K) * 0.125, r(H, K) * 0.125, r(K, H) * 0.011
    y, gate, up = lib().gated_feed_forward_fwd(x, wg, wu, wd, save=True)
    few = lambda t: t[-LAST:].clone()
    y2, gate2, up2 = lib().gated_feed_forward_fwd(few(x), wg, wu, wd, save=True)
    assert torch.equal(gate[-LAST:], gate2) and torch.equal(up[-LAST:], up2)
    off = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())
    assert off(y[-LAST:], y2) <= 2.0 ** -8
    dx = lib().gated_feed_forward_bwd(dy, x, wg, wu, wd, gate, up)[0]
    dx2 = lib().gated_feed_forward_bwd(few(dy), few(x), wg, wu, wd, gate2, up2)[0]
    assert off(dx[-LAST:], dx2) <= 2.0 ** -8
    assert torch.isfinite(dx.float()).all()
