"""Calls from a host thread whose first CUDA call they are."""
import threading

import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu


def test_tensor_maps_on_a_thread_without_a_context():
    gdn = lib()
    entry = gdn._abi_layer.ENTRIES["gdn_linrec_fwd"]
    x, g = torch.randn(1, 300, 64, device="cuda"), -torch.rand(1, 300, 64, device="cuda")
    want, state = gdn.gated_linear_recurrence_fwd(x, g)
    h = torch.empty_like(want)
    torch.cuda.synchronize()
    packed = entry.pack(x.data_ptr(), g.data_ptr(), 0, 0, 0, 1, 300, 64, 1, 0, h.data_ptr(), 0)
    errors = []

    def call():
        try:
            entry(packed, 0, 0, 0)
        except gdn.GdnError as e:
            errors.append(e)

    t = threading.Thread(target=call)
    t.start()
    t.join()
    assert not errors
    torch.cuda.synchronize()
    assert torch.equal(h, want)
