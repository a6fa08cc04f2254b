"""The layer operators as a program uses them: captured in a CUDA graph, their results independent of
what the buffers that they are given held before, and gradients that arrive on any address."""
import contextlib

import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu


def rand(*shape, seed=0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    if isinstance(out, lib().MxTensor):
        return [out.data.view(torch.uint8), out.scales]
    return [t for o in out if o is not None for t in tensors(o)]


def recurrence(B, T, D, lengths=None, dtype=torch.bfloat16):
    if lengths is not None:
        B, T, N = 1, sum(lengths), len(lengths)
        cu = torch.tensor([0] + lengths).cumsum(0).int().cuda()
    else:
        cu, N = None, B
    x, g, dh = (rand(B, T, D, seed=s, dtype=dtype) for s in (1, 2, 3))
    h0, a = rand(N, D, seed=4, dtype=torch.float32), rand(D, seed=5, dtype=torch.float32).abs()

    def run():
        h, ht = lib().gated_linear_recurrence_fwd(x, g, h0, cu, a)
        return h, ht, *lib().gated_linear_recurrence_bwd(dh, g, h, ht, h0, cu, a)
    return run, [x, g, dh]


def step():
    x, g = rand(5, 96, seed=1), rand(5, 96, seed=2)
    state, a = rand(5, 96, seed=3, dtype=torch.float32), rand(96, seed=4, dtype=torch.float32).abs()
    out = torch.empty_like(state)
    return lambda: (lib().gated_linear_recurrence_step(x, g, state, a, out_state=out), out.clone()), [x, g, state]


def norm(rows, D, dtype=torch.bfloat16):
    x, r, dy, dr = (rand(rows, D, seed=s, dtype=dtype) for s in (1, 2, 3, 4))
    w = rand(D, seed=5, dtype=dtype)

    def run():
        y, s, rstd = lib().add_rms_norm_fwd(x, w, r, save_rstd=True)
        out = (y, s, rstd, *lib().add_rms_norm_bwd(dy, s, w, rstd, dr))
        return out if D % 32 else (*out, *lib().add_rms_norm_fwd(x, w, r, out="mxfp8"))
    return run, [x, r, dy, dr]


def product(M, N, K, fmt, dtype=torch.bfloat16):
    x, w = rand(M, K, seed=1, dtype=dtype), lib().mx_quantize(rand(N, K, seed=2), fmt)

    def run():
        q = lib().mx_quantize(x, fmt)
        return lib().mx_linear(x, w), q, lib().mx_dequantize(q), lib().mx_matmul(q, w, torch.float32)
    return run, [x]


CASES = {
    "recurrence in single CTAs": lambda: recurrence(4, 300, 4096),
    "recurrence in clusters": lambda: recurrence(1, 4000, 512, dtype=torch.float32),
    "recurrence in parts": lambda: recurrence(1, 40000, 64),
    "recurrence, packed": lambda: recurrence(0, 0, 200, [5, 0, 300, 1, 700]),
    "recurrence, odd width": lambda: recurrence(2, 500, 67),
    "recurrence, one token": step,
    "norm": lambda: norm(700, 520),
    "norm with MX output": lambda: norm(130, 1056),
    "norm, odd width": lambda: norm(300, 1001, torch.float32),
    "product of few tokens": lambda: product(5, 640, 1024, "mxfp4"),
    "product of a ragged batch": lambda: product(200, 1000, 992, "mxfp8"),
    "large product": lambda: product(1900, 2600, 544, "mxfp4"),
    "product that quantises most rows itself": lambda: product(5200, 4096, 2048, "mxfp8"),
}


@pytest.mark.parametrize("case", list(CASES))
def test_graph_replay_matches_eager_calls(case):
    """Captured once, replayed on other inputs in the same buffers, twice in a row."""
    run, inputs = CASES[case]()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = tensors(run())
    for seed in (7, 8):
        for i, t in enumerate(inputs):
            t.copy_(rand(*t.shape, seed=100 * seed + i, dtype=t.dtype))
        want = tensors(run())
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert len(outs) == len(want) and all(torch.equal(a, b) for a, b in zip(outs, want))
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0


@contextlib.contextmanager
def filled_allocations(byte):
    """Every buffer that the layer operators allocate holds `byte` throughout."""
    from gated_deltanet_linear_bwd_gb300 import layer
    names = ("_empty", "_empty_like")
    real = {n: getattr(layer, n) for n in names}
    made = []

    def filled(make):
        def f(*args, **kw):
            t = make(*args, **kw)
            if t.is_cuda and t.numel() > 0:
                t.view(torch.uint8).fill_(byte)
                made.append(t.numel())
            return t
        return f

    for n in names:
        setattr(layer, n, filled(real[n]))
    try:
        yield made
    finally:
        for n in names:
            setattr(layer, n, real[n])


@pytest.mark.parametrize("case", list(CASES))
def test_results_do_not_depend_on_buffer_contents(case):
    run, _ = CASES[case]()
    results = []
    for byte in (0x00, 0xff):
        with filled_allocations(byte) as made:
            out = run()
        assert len(made) >= 1
        results.append([t.cpu() for t in tensors(out)])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0
