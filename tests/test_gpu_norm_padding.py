"""The MXFP8 norm's scale bytes past the end of the matrix are zeros (2^-127), whatever its rows hold."""
import numpy as np
import pytest
import torch

from gpu_helpers import lib
from layer_ref import tiled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(3, 32), (5, 64), (130, 96), (1, 160), (200, 1056), (2, 4128)])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_scales_past_the_end_are_zeros(eps, rows, D, dtype):
    x = torch.randn(rows, D, generator=torch.Generator().manual_seed(D)).to(dtype).cuda()
    w = torch.ones(D, dtype=dtype, device="cuda")
    x[rows - 1, D // 2] = float("nan")
    if rows > 1:
        x[0] = 0.0                              # with eps = 0 a row of zeros is 0 / 0
    t = lib().add_rms_norm_fwd(x, w, out="mxfp8", eps=eps)[0]
    s = t.scales.cpu().numpy()
    R, B = s.shape[:2]
    byte = s.transpose(0, 3, 2, 1, 4).reshape(128 * R, 4 * B)[:rows, :D // 32]
    assert np.array_equal(s, tiled(byte))       # zeros past the end
    assert (byte[rows - 1] == 255).all()
    if rows > 1:
        assert (byte[0] == (255 if eps == 0 else 0)).all()
    if rows > 2:
        assert (byte[1:rows - 1] < 255).all()
    c = lib().mx_matmul(t, lib().mx_quantize(torch.ones(40, D, device="cuda"), "mxfp8"), torch.float32)
    assert torch.isnan(c[rows - 1]).all() and (rows < 3 or torch.isfinite(c[1:rows - 1]).all())
