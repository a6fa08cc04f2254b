"""Loops and orders that only larger calls run: CTAs of the norm's backward pass that take several rows,
CTAs of the recurrence that walk several sequences one after the other, and products whose tiles go
down the columns first; against 64 bits, with the tolerances of the smaller sizes' tests."""
import numpy as np
import pytest
import torch

import test_gpu_linrec as rec
from gpu_helpers import lib

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def close(name, got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (name, int(bad.sum()), float((got.double() - want).abs().max()))


# more rows than CTAs, in CTAs of several rows, of one, and for rows that are read one by one
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,D", [(5000, 520), (3000, 4096), (4000, 4095), (1300, 16384), (1500, 9001), (20000, 33)])
def test_norm_of_many_rows(rows, D, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows + D)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, r, dy, dr = ((f * rand(rows, D)).to(DT[dtype]) for f in (1, 3, 1, 1))
    w = (1 + 0.2 * rand(D)).to(DT[dtype])
    rel, half = (D.bit_length() + 28) * U, 2.0 ** -8 if dtype == "bf16" else 0.0
    y, s, rstd = lib().add_rms_norm_fwd(x, w, r, eps=1e-5, save_rstd=True)
    sum_ = x.double() + r.double()
    inv = (sum_.square().mean(-1, keepdim=True) + 1e-5) ** -0.5
    want = sum_ * inv * w.double()
    close("y", y, want, (rel + half) * want.abs())
    close("s", s, sum_, (half + U) * sum_.abs())
    close("rstd", rstd, inv[:, 0], rel * inv[:, 0])
    for up in (dr, None):
        ds, dw = lib().add_rms_norm_bwd(dy, s, w, rstd, up)
        xh, wdy = s.double() * rstd.double()[:, None], w.double() * dy.double()
        mean, mag = (wdy * xh).mean(-1, keepdim=True), (wdy * xh).abs().mean(-1, keepdim=True)
        more = up.double() if up is not None else torch.zeros(1, dtype=torch.float64, device="cuda")
        want = rstd.double()[:, None] * (wdy - xh * mean) + more
        parts = rstd.double()[:, None] * (wdy.abs() + xh.abs() * mag) + more.abs()
        close("ds", ds, want, rel * parts + half * want.abs())
        terms = dy.double() * xh
        close("dw", dw, terms.sum(0), (rows.bit_length() + 48) * U * terms.abs().sum(0))
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0


UNEVEN = [(37 * i * i + 11 * i) % 61 for i in range(144)] + [300, 0, 129, 513, 0, 64]


# 150 sequences to 64 clusters of a channel group: TMA rows, and rows that it does not take
@pytest.mark.parametrize("dtype,gated,D", [("bf16", True, 4096), ("fp32", False, 4096), ("bf16", False, 4001),
                                           ("fp32", True, 4001)])
@pytest.mark.parametrize("T", [0, 70])
def test_ctas_that_walk_several_sequences(T, D, gated, dtype):
    p = rec.Problem(150 if T else 0, T, D, dtype, gated, lengths=None if T else UNEVEN, seed=D)
    h, ht = lib().gated_linear_recurrence_fwd(p.x, p.g, p.h0, p.cu, p.scale)
    want, E, want_t, Et = rec.reference_fwd(p)
    rec.close("h", h, want, E, dtype)
    rec.close("final state", ht, want_t, Et, "fp32")
    del want, E
    got = lib().gated_linear_recurrence_bwd(p.dh, p.g, h, p.dht, p.h0, p.cu, p.scale)
    out, err = rec.reference_bwd(p, h)
    for name, t in zip(("dx", "dg", "dh0", "ds"), got):
        rec.close(name, t, out[name], err[name], dtype if name in ("dx", "dg") else "fp32")
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("fmt,M,N,K", [("mxfp8", 512, 33000, 4096), ("mxfp4", 700, 33001, 4128)])
def test_product_of_a_large_weight(fmt, M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(N)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, w = (rand(M, K) * torch.exp(rand(M, 1))).bfloat16(), rand(N, K).bfloat16()
    a, b = lib().mx_quantize(x, fmt), lib().mx_quantize(w, fmt)
    va, vb = lib().mx_dequantize(a).double(), lib().mx_dequantize(b).double()      # exact, tested beside
    want, mag = va @ vb.T, va.abs() @ vb.abs().T
    err = (K / 32 + 2) * 2.0 ** -23 * mag
    close("fp32", lib().mx_matmul(a, b, torch.float32), want, err)
    c = lib().mx_matmul(a, b)
    close("bf16", c, want, err * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs())
    assert torch.equal(lib().mx_linear(x, b), c)
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0
