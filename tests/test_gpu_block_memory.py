"""The state space block's operators as a program uses them: captured in a CUDA graph and replayed on
other inputs, their results independent of what the buffers that they are given held before, and the
same whenever they are asked for."""
import contextlib

import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def rand(*shape, seed=0, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def sequences(B, T, lengths):
    if lengths is None:
        return B, T, B, None
    return 1, sum(lengths), len(lengths), torch.tensor([0] + lengths).cumsum(0).int().cuda()


def convolution(B, T, D, lengths=None, dtype=BF, W=4):
    B, T, N, cu = sequences(B, T, lengths)
    x, dy = (rand(B, T, D, seed=s, dtype=dtype) for s in (1, 2))
    w, b, h0, dht = rand(D, W, seed=3, dtype=dtype), rand(D, seed=4, dtype=dtype), rand(N, W - 1, D, seed=5, dtype=dtype), \
        rand(N, W - 1, D, seed=6, dtype=dtype)

    def run():
        new = torch.empty_like(h0)
        one = lib().causal_convolution_step(h0[:, 0].clone(), w, h0, b, out_state=new)
        return (one, new, *lib().causal_convolution_fwd(x, w, b, h0, cu),
                *lib().causal_convolution_bwd(dy, x, w, b, dht, h0, cu))
    return run, [x, dy, h0]


def scan(B, T, D, S, lengths=None, dtype=BF, gate=True):
    B, T, N, cu = sequences(B, T, lengths)
    x, dt, z, dy = (rand(B, T, D, seed=s, dtype=dtype) for s in (1, 2, 3, 4))
    b, c = (rand(B, T, S, seed=s, dtype=dtype) for s in (5, 6))
    a, skip, bias = -rand(D, S, seed=7, dtype=F).abs(), rand(D, seed=8, dtype=F), rand(D, seed=9, dtype=F) - 2
    h0, dht = rand(N, D, S, seed=10, dtype=F), rand(N, D, S, seed=11, dtype=F)
    few = dict(skip=skip, z=z if gate else None, dt_bias=bias, initial_state=h0, cu_seqlens=cu)

    def run():
        new = torch.empty_like(h0)
        token = [t.flatten(0, 1)[:1].repeat(N, 1) for t in (x, dt, b, c)]
        one = lib().state_space_step(token[0], token[1], a, *token[2:], h0, skip, None, bias, out_state=new)
        return (one, new, *lib().state_space_scan_fwd(x, dt, a, b, c, **few),
                *lib().state_space_scan_bwd(dy, x, dt, a, b, c, dht=dht, **few))
    return run, [x, dt, dy, b, c]


def feed_forward(M, K, H):
    x, dy = rand(M, K, seed=1), rand(M, K, seed=2)
    wg, wu, wd = rand(H, K, seed=3) * K ** -0.5, rand(H, K, seed=4) * K ** -0.5, rand(K, H, seed=5) * H ** -0.5

    def run():
        y, gate, up = lib().gated_feed_forward_fwd(x, wg, wu, wd, save=True)
        return (y, gate, up, *lib().gated_feed_forward_bwd(dy, x, wg, wu, wd, gate, up))
    return run, [x, dy]


CASES = {
    "convolution": lambda: convolution(3, 500, 264),
    "convolution, packed": lambda: convolution(0, 0, 130, [5, 0, 300, 1, 2, 64], F, 3),
    "convolution, odd width": lambda: convolution(2, 70, 67, W=2),
    "scan": lambda: scan(20, 150, 2048, 16),
    "scan in parts": lambda: scan(1, 4000, 72, 16),
    "scan in parts, packed": lambda: scan(0, 0, 40, 24, [5, 0, 1500, 1, 700], gate=False),
    "scan, odd width": lambda: scan(2, 100, 33, 5, dtype=F),
    "scan of many states": lambda: scan(0, 0, 96, 64, [40, 3, 0, 33]),
    "feed-forward, few tokens": lambda: feed_forward(5, 520, 1032),
    "feed-forward, a few more": lambda: feed_forward(40, 264, 2056),
    "feed-forward, narrow pairs": lambda: feed_forward(900, 2056, 1000),
    "feed-forward, pairs": lambda: feed_forward(2600, 2056, 2056),
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
        outs = [t for t in run() if t is not None]
    for seed in (7, 8):
        for i, t in enumerate(inputs):
            t.copy_(rand(*t.shape, seed=100 * seed + i, dtype=t.dtype))
        want = [t for t in run() if t is not None]
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert len(outs) == len(want) and all(torch.equal(a, b) for a, b in zip(outs, want))
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0


@contextlib.contextmanager
def filled_allocations(byte):
    """Every buffer that the operators allocate holds `byte` throughout."""
    from gated_deltanet_linear_bwd_gb300 import feed_forward as ff, layer, state_space
    modules, names, made = (layer, state_space, ff), ("_empty", "_empty_like"), []
    real = {(m, n): getattr(m, n) for m in modules for n in names}

    def filled(make):
        def f(*args, **kw):
            t = make(*args, **kw)
            if t.is_cuda and t.numel() > 0:
                t.view(torch.uint8).fill_(byte)
                made.append(t.numel())
            return t
        return f

    for (m, n), f in real.items():
        setattr(m, n, filled(f))
    try:
        yield made
    finally:
        for (m, n), f in real.items():
            setattr(m, n, f)


@pytest.mark.parametrize("case", list(CASES))
def test_results_do_not_depend_on_buffer_contents(case):
    run, _ = CASES[case]()
    results = []
    for byte in (0x00, 0xff):
        with filled_allocations(byte) as made:
            out = run()
        assert len(made) >= 6
        results.append([t.cpu() for t in out if t is not None])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert all(torch.isfinite(t.float()).all() for t in results[0])
    assert lib().gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0


def test_calls_on_two_streams_at_once():
    """Each call has its own workspace: two at once give what they give one after the other."""
    cases = [CASES[c]() for c in ("scan in parts", "feed-forward, a few more", "convolution")]
    want = [[t.clone() for t in run() if t is not None] for run, _ in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(6)]
    for _ in range(5):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append([t for t in cases[i % 3][0]() if t is not None])
        torch.cuda.synchronize()
        for i, out in enumerate(got):
            assert all(torch.equal(a, b) for a, b in zip(out, want[i % 3]))
