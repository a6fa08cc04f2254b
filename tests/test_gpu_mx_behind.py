"""Products right behind kernels that hold all of an SM's tensor memory, and the other way round: the
delta rule's walks and products of already quantised matrices, of a K so short that a CTA of theirs
needs little of an SM, one after the other in one stream."""
import pytest
import torch

import gdn_synth
from gpu_helpers import lib

pytestmark = pytest.mark.gpu


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("M,N,K", [(8, 1280, 64), (64, 9728, 64), (128, 2432, 256), (300, 515, 96), (2048, 2056, 64)])
def test_products_behind_the_delta_rule(M, N, K):
    gdn = lib()
    d = gdn_synth.make("training", B=1, T=512, H=160).to("cuda")
    a, b = gdn.mx_quantize(rand(M, K, seed=1), "mxfp8"), gdn.mx_quantize(rand(N, K, seed=2), "mxfp8")
    want, want_o = gdn.mx_matmul(a, b), gdn.chunk_gated_delta_rule_fwd(d.q, d.k, d.v, d.g, d.beta)[0]
    torch.cuda.synchronize()
    for _ in range(10):
        o = gdn.chunk_gated_delta_rule_fwd(d.q, d.k, d.v, d.g, d.beta)[0]
        c = gdn.mx_matmul(a, b)
        grads = gdn.chunk_gated_delta_rule_bwd(d.q, d.k, d.v, d.g, d.beta, want_o)
        e = gdn.mx_matmul(a, b)
        assert torch.equal(c, want) and torch.equal(e, want) and torch.equal(o, want_o)
    assert all(torch.isfinite(t).all() for t in grads if t is not None)
    assert gdn.gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0


def test_clusters_of_several_streams_share_the_tensor_memory():
    """Products whose CTAs share K in clusters, of every tile width, on four streams at once, with
    a K so short that many of their CTAs would fit an SM."""
    gdn = lib()
    sizes = [(128, 4096, 512), (64, 4096, 512), (20, 4096, 1024), (100, 2432, 640), (10, 1024, 1024), (33, 4864, 512)]
    pairs = [(gdn.mx_quantize(rand(M, K, seed=M), "mxfp8"), gdn.mx_quantize(rand(N, K, seed=N + K), "mxfp8"))
             for M, N, K in sizes]
    want = [gdn.mx_matmul(a, b) for a, b in pairs]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for turn in range(40):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                k = (turn * (i + 1) + i) % len(sizes)
                got.append((k, gdn.mx_matmul(*pairs[k])))
    torch.cuda.synchronize()
    assert all(torch.equal(c, want[k]) for k, c in got)
    assert gdn.gdn_sync_status(torch.cuda.current_stream().cuda_stream) == 0
