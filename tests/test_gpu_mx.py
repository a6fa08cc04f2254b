"""Microscaled quantisation (bit for bit) and product, against 64 bits.

The product's tolerance: an MMA adds 32 (MXFP8) or 64 (MXFP4) products to an fp32
sum; taking every addition of the K / 32 partial sums as truncated to 24 bits, a
result is off by at most (K / 32 + 2) 2^-23 sum |a b|; a bf16 result, of 8 significant
bits, adds 2^-8 of itself (and 2^-8 of that error)."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from gpu_helpers import lib

pytestmark = pytest.mark.gpu
FMT = ["mxfp8", "mxfp4"]
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def draw(rows, K, seed, dtype="bf16"):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=gen) * torch.exp(2 * torch.randn(rows, 1, generator=gen))
    return x.to(DT[dtype]).cuda()


def codes(t):
    d = t.data.view(torch.uint8).cpu().numpy()
    return d if t.fmt == "mxfp8" else np.stack([d & 15, d >> 4], -1).reshape(d.shape[0], -1)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (33, 96), (127, 128), (130, 160), (200, 1024),
                                    (5, 4096), (1, 8224), (300, 256)])
def test_quantise_bit_for_bit(rows, K, dtype, fmt):
    x = draw(rows, K, rows + K, dtype)
    t = lib().mx_quantize(x, fmt)
    value, byte, code = ref.quantize(x.double().cpu().numpy(), fmt)
    assert np.array_equal(t.scales.cpu().numpy(), ref.tiled(byte))
    assert np.array_equal(codes(t), code)
    want = ref.values(value, byte)
    for dt in DT.values():
        got = lib().mx_dequantize(t, dt).double().cpu().numpy()
        assert np.array_equal(got, want)         # elements of 8 bits times powers of two: exact


@pytest.mark.parametrize("fmt", FMT)
def test_quantise_special_values(fmt):
    """Ties, the largest element and just past it, zeros, subnormal and huge values, NaN, infinities."""
    top = ref.GRID[fmt][-1]
    rows = []
    for s in (1.0, 2.0 ** -100, 2.0 ** 100):
        mid = (ref.GRID[fmt][:-1] + ref.GRID[fmt][1:]) / 2
        for k in range(0, len(mid), 15):
            rows.append(np.concatenate([[top], mid[k:k + 15], -mid[k:k + 15], np.zeros(32)])[:32] * s)
        for big in (top, np.nextafter(np.float32(top), np.float32(1e9)), np.nextafter(np.float32(top), np.float32(0))):
            rows.append(np.concatenate([[big], np.linspace(-1, 1, 31)]) * s)
    rows.append(np.zeros(32))
    rows.append(np.full(32, -0.0))
    rows.append(np.linspace(-1, 1, 32) * 1e-40)
    rows.append(np.linspace(-1, 1, 32) * 2.0 ** -126)
    rows.append(np.linspace(-1, 1, 32) * 3.4e38)
    for bad in (np.nan, np.inf, -np.inf):
        rows.append(np.concatenate([[1.0, bad], np.ones(30)]))
    x = torch.tensor(np.array(rows, dtype=np.float32)).cuda()
    t = lib().mx_quantize(x, fmt)
    value, byte, code = ref.quantize(x.double().cpu().numpy(), fmt)
    assert np.array_equal(t.scales.cpu().numpy(), ref.tiled(byte))
    assert np.array_equal(codes(t), code)
    got = lib().mx_dequantize(t).cpu().numpy()
    with np.errstate(over="ignore"):
        want = ref.values(value, byte).astype(np.float32)
    assert np.array_equal(got, want, equal_nan=True)


def reference_product(a, b):
    a, b = (torch.from_numpy(ref.values(*v[:2])).cuda() for v in (a, b))
    return (a @ b.T).cpu().numpy(), (a.abs() @ b.abs().T).cpu().numpy()


SIZES = [(1, 1, 32), (1, 128, 32), (3, 5, 64), (7, 129, 96), (16, 300, 160), (17, 64, 4096), (31, 1000, 992),
         (64, 513, 544), (65, 256, 512), (128, 128, 256), (129, 130, 288), (200, 77, 1056), (1000, 520, 320),
         (257, 640, 2080), (512, 1024, 1024), (4, 4096, 4096), (300, 515, 8192),
         # enough tiles for CTA pairs: whole, ragged rows, columns and K, several tiles to a pair
         (2048, 2048, 512), (2500, 2568, 544), (1900, 5000, 96), (4097, 3336, 32), (2300, 2056, 1056)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, fmt):
    x, w = draw(M, K, M + K), draw(N, K, N + K + 1)
    a, b = lib().mx_quantize(x, fmt), lib().mx_quantize(w, fmt)
    qa, qb = (ref.quantize(v.double().cpu().numpy(), fmt) for v in (x, w))
    want, mag = reference_product(qa, qb)
    err = (K / 32 + 2) * 2.0 ** -23 * mag
    for dt, extra in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
        got = lib().mx_matmul(a, b, dt).double().cpu().numpy()
        bad = ~(np.abs(got - want) <= err * (1 + extra) + extra * np.abs(want))
        assert not bad.any(), (int(bad.sum()), float(np.abs(got - want).max()), float(err.max()))
    assert torch.equal(lib().mx_linear(x, b), lib().mx_matmul(a, b))
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("fmt", FMT)
def test_product_of_units_places_every_element(fmt):
    """Rows of the identity against a matrix whose values name their place: each result is one
    element, exactly."""
    K = N = 320
    eye = torch.eye(K, device="cuda")
    w = (torch.arange(N, device="cuda")[:, None] % 7 - 3) * 2.0 ** (torch.arange(K, device="cuda")[None] // 32 % 9 - 4)
    a, b = lib().mx_quantize(eye, fmt), lib().mx_quantize(w, fmt)
    assert torch.equal(lib().mx_dequantize(b), w)
    assert torch.equal(lib().mx_matmul(a, b, torch.float32), w.T)
    assert torch.equal(lib().mx_matmul(b, a, torch.float32), w)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,N", [(5, 200), (150, 200), (600, 200), (2100, 2400)])
def test_nan_blocks_reach_their_row_only(fmt, M, N):
    x, w = draw(M, 256, 1), draw(N, 256, 2)
    clean = lib().mx_matmul(lib().mx_quantize(x, fmt), lib().mx_quantize(w, fmt))
    x[3, 40] = float("inf")
    w[7, 3] = float("nan")
    c = lib().mx_linear(x, lib().mx_quantize(w, fmt))
    assert torch.isnan(c[3]).all() and torch.isnan(c[:, 7]).all()
    keep = torch.ones_like(c, dtype=torch.bool)
    keep[3], keep[:, 7] = False, False
    assert torch.equal(c[keep], clean[keep])


def test_none_of_something():
    for M, N, K in ((0, 8, 64), (8, 0, 64), (4, 8, 0)):
        a, b = (lib().mx_quantize(torch.ones(r, K, device="cuda"), "mxfp8") if r and K else
                lib().MxTensor.empty(r, K, "mxfp8", "cuda") for r in (M, N))
        c = lib().mx_matmul(a, b)
        assert c.shape == (M, N) and not c.any()


@pytest.mark.parametrize("fmt", FMT)
def test_checkpoint_parts_and_leading_axes(fmt):
    w = draw(140, 96, 5)
    value, byte, _ = ref.quantize(w.double().cpu().numpy(), fmt)
    t = lib().mx_quantize(w, fmt)
    again = lib().mx_from_parts(t.data.clone(), torch.tensor(byte, dtype=torch.uint8).cuda(), fmt)
    assert torch.equal(again.scales, t.scales)
    x = draw(12, 96, 6)
    y = lib().mx_linear(x.view(3, 4, 96), again)
    assert y.shape == (3, 4, 140) and torch.equal(y.view(12, 140), lib().mx_linear(x, t))


@pytest.mark.parametrize("fmt", FMT)
def test_repeats_bit_for_bit_and_on_another_stream(fmt):
    for M, N in ((4, 640), (300, 640), (3000, 2048)):
        x, w = draw(M, 4096, 1), lib().mx_quantize(draw(N, 4096, 2), fmt)
        first = lib().mx_linear(x, w)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            with torch.cuda.stream(side):
                again = lib().mx_linear(x, w)
            side.synchronize()
            assert torch.equal(first, again)


@pytest.mark.parametrize("M", [4, 3000])
def test_bounded_waits_give_up_and_the_next_call_is_right(M):
    x, w = draw(M, 1024, 1), lib().mx_quantize(draw(2048, 1024, 2), "mxfp8")
    a = lib().mx_quantize(x, "mxfp8")
    want = lib().mx_matmul(a, w)
    stream = torch.cuda.current_stream().cuda_stream
    try:
        lib().gdn_set_spin_limit(0)
        lib().mx_matmul(a, w)
        assert lib().gdn_sync_status(stream) == 5
    finally:
        lib().gdn_set_spin_limit(-1)
    assert torch.equal(lib().mx_matmul(a, w), want)
    assert lib().gdn_sync_status(stream) == 0


def test_refusals():
    q, mm = lib().mx_quantize, lib().mx_matmul
    x = draw(8, 64, 1)
    a8, a4 = q(x, "mxfp8"), q(x, "mxfp4")
    other = q(draw(8, 96, 1), "mxfp8")
    for bad in (lambda: q(x.cpu()), lambda: q(x, "int4"), lambda: q(x[:, :40].contiguous()),
                lambda: q(x[:, ::2]), lambda: q(x.half()), lambda: mm(a8, a4), lambda: mm(a8, other),
                lambda: mm(x, a8), lambda: lib().MxTensor(a8.data, a8.scales.flatten()[:100], "mxfp8", (8, 64)),
                lambda: lib().MxTensor(a8.data, a8.scales, "mxfp4", (8, 64)),
                lambda: lib().mx_from_parts(a8.data, torch.zeros(8, 3, dtype=torch.uint8, device="cuda"), "mxfp8"), lambda: mm(a8, a8, torch.float16),
                lambda: lib().mx_linear(x, other), lambda: lib().mx_dequantize(a8, torch.float16)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lib().GdnError, match="aligned"):
        q(torch.zeros(1 + 64, device="cuda")[1:].view(1, 64))


# mx_linear of sizes at which the product quantises most rows itself: whole and ragged tiles of
# rows, an odd number of 128-row blocks, K of several strips and of a part of one, either type
FUSED = [(5200, 4096, 2048), (5376, 4104, 4160), (3201, 8200, 2080), (5150, 4360, 8352), (5130, 4099, 2048)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,N,K", FUSED)
def test_linear_is_quantisation_and_product(M, N, K, fmt, dtype):
    x, w = draw(M, K, 7).to(DT[dtype]), lib().mx_quantize(draw(N, K, 8), fmt)
    x[M - 3, 40], x[300, 5] = float("nan"), float("inf")
    want = lib().mx_matmul(lib().mx_quantize(x, fmt), w, DT[dtype])
    assert torch.isnan(want[M - 3]).all() and torch.isnan(want[300]).all()
    for _ in range(3):
        assert torch.equal(lib().mx_linear(x, w).nan_to_num(7.0), want.nan_to_num(7.0))
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0


def test_linear_on_two_streams_at_once():
    xs = [draw(4096, 2048, s) for s in (1, 2)]
    w = lib().mx_quantize(draw(4104, 2048, 3), "mxfp8")
    want = [lib().mx_matmul(lib().mx_quantize(x, "mxfp8"), w) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(lib().mx_linear(xs[i], w))
    torch.cuda.synchronize()
    assert all(torch.equal(c, want[i]) for i in (0, 1) for c in got[i])


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,N,K", [(2048, 2049, 512), (2307, 2571, 544), (1900, 5003, 96), (700, 12290, 288), (4097, 3337, 32)])
def test_large_products_of_odd_widths(M, N, K, fmt):
    """Rows of C that start on no 16 bytes (bf16 and fp32), from the kernel of large products."""
    test_product(M, N, K, fmt)
    x, w = draw(M, K, 1), lib().mx_quantize(draw(N, K, 2), fmt)
    wide = lib().mx_quantize(draw(N, K, 2)[:N - N % 8], fmt)          # a width that TMA stores
    a = lib().mx_quantize(x, fmt)
    for dt in DT.values():
        assert torch.equal(lib().mx_matmul(a, w, dt)[:, :N - N % 8], lib().mx_matmul(a, wide, dt))


@pytest.mark.parametrize("fmt", FMT)
def test_linear_whose_waits_give_up_and_the_next_call_is_right(fmt):
    x, w = draw(5200, 2048, 1), lib().mx_quantize(draw(4096, 2048, 2), fmt)
    want = lib().mx_matmul(lib().mx_quantize(x, fmt), w)
    stream = torch.cuda.current_stream().cuda_stream
    try:
        lib().gdn_set_spin_limit(0)
        lib().mx_linear(x, w)
        assert lib().gdn_sync_status(stream) == 5
    finally:
        lib().gdn_set_spin_limit(-1)
    assert torch.equal(lib().mx_linear(x, w), want)
    assert lib().gdn_sync_status(stream) == 0
