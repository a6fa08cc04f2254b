"""Residual addition with the RMS norm, forward (plain and MXFP8) and backward, in
64 bits.

Tolerances, u = 2^-24.  rstd: a sum of D squares in at most 16 + log2(D) + 2 dependent
additions, a division and rsqrt (2 ulp): (D.bit_length() + 24) u relative.  y adds three
products: (D.bit_length() + 28) u of itself, and 2^-8 of itself in bf16 (8 significant bits).  MXFP8: an element may differ from the reference's by one grid step where the
scaled value lies within that error of the middle between two, and a scale by one power of two
where the largest value does; so the dequantised values may be off by half a step of the coarser
grid plus that error: 2^-4 of the value plus 2^-10 of the block's scale, times (1 + 1e-4).
Backward: the row's mean of w dy xh carries (D.bit_length() + 28) u of the mean of magnitudes; dw's
sum over rows (bit_length(rows) + 40) u of the sum of magnitudes, plus 8 u of each term."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from gpu_helpers import lib

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
SHAPES = [(1, 1), (3, 7), (5, 32), (2, 33), (300, 64), (1, 100), (9, 129), (130, 256), (17, 1000), (4, 2048), (3, 4096),
          (700, 520), (2, 5001), (3, 8192), (2, 16384)]


def draw(rows, D, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    return [(t * f).to(DT[dtype]).cuda() for t, f in ((r(rows, D), 1), (r(rows, D), 3), (r(rows, D), 1),
                                                      (r(rows, D), 1), (1 + 0.2 * r(D), 1))]


def np64(t):
    return t.double().cpu().numpy()


def close(got, want, tol):
    bad = ~(np.abs(np64(got) - want) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.abs(np64(got) - want).max()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_forward_and_backward(rows, D, dtype):
    x, r, dy, dr, w = draw(rows, D, dtype, rows + D)
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    rel = (D.bit_length() + 28) * U
    for res in (r, None):
        s = np64(x) + (np64(res) if res is not None else 0)
        rstd = (np.mean(s * s, -1, keepdims=True) + 1e-5) ** -0.5
        y, got_s, got_r = lib().add_rms_norm_fwd(x, w, res, eps=1e-5, save_rstd=True)
        close(y, s * rstd * np64(w), (rel + half) * np.abs(s * rstd * np64(w)))
        close(got_s, s, (half + U) * np.abs(s))
        close(got_r, rstd[:, 0], rel * rstd[:, 0])
        assert lib().add_rms_norm_fwd(x, w, res, eps=1e-5)[2] is None

        # the backward's own definition, from the stored s and rstd
        s, rstd = np64(got_s), np64(got_r)[:, None]
        for up in (dr, None):
            ds, dw = lib().add_rms_norm_bwd(dy, got_s, w, got_r, up)
            xh, wdy = s * rstd, np64(w) * np64(dy)
            mean, mag = (wdy * xh).mean(-1, keepdims=True), np.abs(wdy * xh).mean(-1, keepdims=True)
            want = rstd * (wdy - xh * mean) + (np64(up) if up is not None else 0)
            parts = rstd * (np.abs(wdy) + np.abs(xh) * mag) + (np.abs(np64(up)) if up is not None else 0)
            close(ds, want, rel * parts + half * np.abs(want))
            terms = np.abs(np64(dy) * xh)
            close(dw, (np64(dy) * xh).sum(0), (rows.bit_length() + 48) * U * terms.sum(0))
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0


def untile(scales, rows, blocks):
    t = scales.cpu().numpy().astype(int)
    R, B = t.shape[:2]
    return t.transpose(0, 3, 2, 1, 4).reshape(128 * R, 4 * B)[:rows, :blocks]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,D", [(1, 32), (3, 64), (130, 96), (129, 160), (300, 256), (40, 1024), (5, 4096),
                                    (3, 8192), (2, 16384), (2000, 128)])
def test_mx_output(rows, D, dtype):
    x, r, _, _, w = draw(rows, D, dtype, rows + D)
    for res in (r, None):
        s = np64(x) + (np64(res) if res is not None else 0)
        y = s * (np.mean(s * s, -1, keepdims=True) + 1e-6) ** -0.5 * np64(w)
        t, got_s, _ = lib().add_rms_norm_fwd(x, w, res, out="mxfp8")
        byte = untile(t.scales, rows, D // 32)
        _, want_byte, _ = ref.quantize(y, "mxfp8")
        assert (np.abs(byte - want_byte) <= 1).all() and (byte != want_byte).mean() <= 0.01
        tiles = t.scales.cpu().numpy()
        assert np.array_equal(tiles, ref.tiled(byte))          # zeros past the end
        got = np64(lib().mx_dequantize(t))
        scale = np.repeat(2.0 ** (np.maximum(byte, want_byte) - 127.0), 32, -1)
        assert (np.abs(got - y) <= (2.0 ** -4 * np.abs(y) + 2.0 ** -10 * scale) * (1 + 1e-4)).all()
        # and as the quantised plain output, but for the rare element on a rounding's edge
        plain = lib().add_rms_norm_fwd(x.float(), w.float(), None if res is None else res.float())[0]
        q = lib().mx_quantize(plain, "mxfp8")
        assert (q.data.view(torch.uint8) != t.data.view(torch.uint8)).float().mean() <= 0.01
        close(got_s, s, (2.0 ** -8 if dtype == "bf16" else U) * np.abs(s))


def test_rows_without_size_and_bad_values():
    x, r, dy, dr, w = draw(6, 256, "fp32", 1)
    x[0], x[1, 3], x[2, 5] = 0, float("nan"), float("inf")
    x[3] *= 1e-25                                   # squares that underflow: eps alone is left
    y, s, rstd = lib().add_rms_norm_fwd(x, w, save_rstd=True)
    assert not y[0].any() and torch.isnan(y[1]).all() and torch.isfinite(y[3:]).all()
    assert torch.allclose(y[3], x[3] * 1e3 * w, rtol=1e-5)
    assert torch.isnan(y[2, 5]) and not y[2, :5].any()
    t = lib().add_rms_norm_fwd(x, w, out="mxfp8")[0]
    byte = untile(t.scales, 6, 8)
    assert not byte[0].any() and (byte[1] == 255).all() and byte[2, 0] == 255 and not byte[2, 1:].any()
    d = lib().mx_dequantize(t)
    assert torch.isnan(d[1]).all() and torch.isfinite(d[[0, 3, 4, 5]]).all()


def test_more_than_2_to_31_elements():
    rows, D = 300_000, 8192
    x = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    y = lib().add_rms_norm_fwd(x, w)[0]
    assert torch.equal(y[-5:], lib().add_rms_norm_fwd(x[-5:].clone(), w)[0])
    t = lib().add_rms_norm_fwd(x, w, x, out="mxfp8")[0]
    u = lib().add_rms_norm_fwd(x[-32:].clone(), w, x[-32:].clone(), out="mxfp8")[0]
    assert torch.equal(t.data[-32:].view(torch.uint8), u.data.view(torch.uint8))
    q = lib().mx_quantize(x, "mxfp4")
    assert torch.equal(q.data[-32:], lib().mx_quantize(x[-32:].clone(), "mxfp4").data)


def test_gradients_match_central_differences():
    """fp32, along random directions, step 1e-2: rounding of a sum of ~100 terms of size ~3 gives
    100 * 3 * 2^-24 / 1e-2 = 2e-3 of scale 1; 5e-3 of the gradient's and direction's norms allowed."""
    x, r, dy, dr, w = draw(3, 40, "fp32", 2)
    ins = [t.requires_grad_() for t in (x, w, r)]

    def f(x, w, r):
        y, s = lib().add_rms_norm(x, w, r)
        return (y.double() * dy).sum() + (s.double() * dr).sum()

    grads = torch.autograd.grad(f(*ins), ins)
    gen = torch.Generator().manual_seed(5)
    for k, grad in enumerate(grads):
        d = torch.randn(grad.shape, generator=gen).cuda()
        with torch.no_grad():
            up, down = ([t + sign * 1e-2 * d if j == k else t for j, t in enumerate(ins)] for sign in (1, -1))
            num = float((f(*up) - f(*down)) / 2e-2)
        scale = float(grad.double().norm() * d.double().norm())
        assert abs(num - float((grad.double() * d).sum())) <= 5e-3 * scale
    y = lib().add_rms_norm(x, w)
    (g,) = torch.autograd.grad((y * dy).sum(), x)
    assert torch.isfinite(g).all()


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    assert lib().add_rms_norm_fwd(x, w)[0].shape == (0, 64)
    ds, dw = lib().add_rms_norm_bwd(x, x, w, torch.empty(0, device="cuda"))
    assert ds.shape == (0, 64) and not dw.any()
    assert lib().add_rms_norm_fwd(x, w, out="mxfp8")[0].data.shape == (0, 64)


def test_repeats_bit_for_bit_and_on_another_stream():
    x, r, dy, dr, w = draw(1000, 520, "bf16", 3)
    run = lambda: (*lib().add_rms_norm_fwd(x, w, r, save_rstd=True), *lib().add_rms_norm_bwd(dy, x, w, rstd, dr))
    rstd = lib().add_rms_norm_fwd(x, w, save_rstd=True)[2]
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(side):
            again = run()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_refusals():
    x, r, dy, dr, w = draw(4, 64, "bf16", 3)
    f, b = lib().add_rms_norm_fwd, lib().add_rms_norm_bwd
    rstd = torch.ones(4, device="cuda")
    for bad in (lambda: f(x.cpu(), w), lambda: f(x, w.float()), lambda: f(x, w[:32].contiguous()), lambda: f(x.half(), w),
                lambda: f(x, w, r[:2].contiguous()), lambda: f(x[:, ::2], w[::2].contiguous()), lambda: f(x, w, out="int8"),
                lambda: f(x[:, :40].contiguous(), w[:40].contiguous(), out="mxfp8"),
                lambda: b(dy, x, w, rstd[:2]), lambda: b(dy, x.float(), w, rstd),
                lambda: b(dy, x, w, rstd, dr[:, :32].contiguous())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lib().GdnError, match="16384"):
        f(torch.zeros(1, 16400, device="cuda"), torch.zeros(16400, device="cuda"))
