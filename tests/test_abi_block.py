"""The C ABI of the block operators without a GPU: host-side refusals, workspaces, empty problems."""
import pytest

from test_abi_layer import abi  # noqa: F401  (a fixture)

TOP = 2 ** 31 - 1
OK = dict(
    gdn_conv_fwd=dict(x=4096, weight=4096, y=4096, B=2, T=5, D=64, W=4),
    gdn_conv_bwd=dict(d_y=4096, x=4096, weight=4096, dx=4096, dweight=4096, B=2, T=5, D=64, W=4),
    gdn_conv_step=dict(x=4096, weight=4096, state=4096, y=4096, out_state=4096, N=2, D=64, W=4),
    gdn_ssm_fwd=dict(x=4096, dt=4096, a=4096, b=4096, c=4096, y=4096, B=1, T=5000, D=64, S=16),
    gdn_ssm_bwd=dict(d_y=4096, x=4096, dt=4096, a=4096, b=4096, c=4096, dx=4096, ddt=4096, da=4096, db=4096, dc=4096,
                     B=2, T=5, D=64, S=16),
    gdn_ssm_step=dict(x=4096, dt=4096, a=4096, b=4096, c=4096, state=4096, y=4096, out_state=4096, N=2, D=64, S=16),
    gdn_ffn_fwd=dict(x=4096, w_gate=4096, w_up=4096, w_down=4096, y=4096, M=3, K=64, F=128, dtype=1, activation=1),
    gdn_ffn_bwd=dict(d_y=4096, x=4096, w_gate=4096, w_up=4096, w_down=4096, gate=4096, up=4096, dx=4096, dw_gate=4096,
                     dw_up=4096, dw_down=4096, M=3, K=64, F=128, dtype=1, activation=1),
)


def raw(abi, name, **kw):
    a = getattr(abi, name + "_args")()
    for k, v in {**OK[name], **kw}.items():
        setattr(a, k, v)
    return bytes(a)


def call(abi, name, **kw):
    args = raw(abi, name, **kw)
    f = getattr(abi.load(), name)
    return f(args, 4096, 1 << 40, None) if name + "_workspace_size" in abi.EXPORTS else f(args, None)


@pytest.mark.parametrize("name, bad, rc, msg", [
    ("gdn_conv_fwd", dict(B=0), 1, "bad sizes"),
    ("gdn_conv_fwd", dict(T=-1), 1, "bad sizes"),
    ("gdn_conv_fwd", dict(D=0), 1, "bad sizes"),
    ("gdn_conv_fwd", dict(W=1), 2, "W = 1"),
    ("gdn_conv_fwd", dict(W=5), 2, "W = 5"),
    ("gdn_conv_fwd", dict(dtype=2), 2, "dtype"),
    ("gdn_conv_fwd", dict(activation=2), 2, "activation"),
    ("gdn_conv_fwd", dict(weight=None), 1, "required"),
    ("gdn_conv_fwd", dict(y=None), 1, "required"),
    ("gdn_conv_fwd", dict(x=4104), 1, "aligned"),
    ("gdn_conv_fwd", dict(final_state=4098), 1, "aligned"),
    ("gdn_conv_fwd", dict(cu_seqlens=4096, N=1), 1, "cu_seqlens"),
    ("gdn_conv_fwd", dict(cu_seqlens=4096, B=1, N=0), 1, "cu_seqlens"),
    ("gdn_conv_fwd", dict(B=1 << 16, T=1 << 16), 1, "too large"),
    ("gdn_conv_fwd", dict(D=TOP), 1, "too large"),
    ("gdn_conv_fwd", dict(cu_seqlens=4096, B=1, N=TOP), 1, "too large"),
    ("gdn_conv_bwd", dict(dweight=None), 1, "required"),
    ("gdn_conv_bwd", dict(d_y=None), 1, "required"),
    ("gdn_conv_bwd", dict(dbias=4100), 1, "aligned"),
    ("gdn_conv_bwd", dict(W=0), 2, "W = 0"),
    ("gdn_conv_step", dict(N=-1), 1, "bad sizes"),
    ("gdn_conv_step", dict(state=None), 1, "required"),
    ("gdn_conv_step", dict(out_state=4100), 1, "aligned"),
    ("gdn_conv_step", dict(activation=3), 2, "activation"),
    ("gdn_ssm_fwd", dict(S=0), 1, "bad sizes"),
    ("gdn_ssm_fwd", dict(S=65), 2, "S = 65"),
    ("gdn_ssm_fwd", dict(T=-1), 1, "bad sizes"),
    ("gdn_ssm_fwd", dict(dtype=3), 2, "dtype"),
    ("gdn_ssm_fwd", dict(a=None), 1, "required"),
    ("gdn_ssm_fwd", dict(c=None), 1, "required"),
    ("gdn_ssm_fwd", dict(z=4104), 1, "aligned"),
    ("gdn_ssm_fwd", dict(cu_seqlens=4096, B=2, N=1), 1, "cu_seqlens"),
    ("gdn_ssm_fwd", dict(B=70000), 1, "too large"),
    ("gdn_ssm_fwd", dict(T=TOP), 1, "too large"),
    ("gdn_ssm_fwd", dict(T=1 << 30, D=1 << 20), 1, "too large"),
    ("gdn_ssm_bwd", dict(da=None), 1, "required"),
    ("gdn_ssm_bwd", dict(z=4096), 1, "required"),
    ("gdn_ssm_bwd", dict(d_final_state=4100), 1, "aligned"),
    ("gdn_ssm_step", dict(N=-1), 1, "bad sizes"),
    ("gdn_ssm_step", dict(out_state=None), 1, "required"),
    ("gdn_ssm_step", dict(state=4104), 1, "aligned"),
    ("gdn_ssm_step", dict(N=TOP), 1, "too large"),
    ("gdn_ffn_fwd", dict(M=-1), 1, "bad sizes"),
    ("gdn_ffn_fwd", dict(K=0), 1, "bad sizes"),
    ("gdn_ffn_fwd", dict(K=60), 2, "multiples of 8"),
    ("gdn_ffn_fwd", dict(F=100), 2, "multiples of 8"),
    ("gdn_ffn_fwd", dict(F=TOP), 1, "too large"),
    ("gdn_ffn_fwd", dict(dtype=0), 2, "dtype"),
    ("gdn_ffn_fwd", dict(activation=0), 2, "activation"),
    ("gdn_ffn_fwd", dict(gate=4096), 1, "together"),
    ("gdn_ffn_fwd", dict(w_down=None), 1, "required"),
    ("gdn_ffn_fwd", dict(y=4104), 1, "aligned"),
    ("gdn_ffn_bwd", dict(dw_up=None), 1, "required"),
    ("gdn_ffn_bwd", dict(up=None), 1, "required"),
    ("gdn_ffn_bwd", dict(dx=4100), 1, "aligned"),
    ("gdn_ffn_bwd", dict(activation=7), 2, "activation"),
])
def test_bad_arguments_are_rejected_on_the_host(abi, name, bad, rc, msg):
    assert call(abi, name, **bad) == rc
    assert msg in abi._abi.gdn_last_error()


def test_null_arguments_and_small_workspaces(abi):
    lib = abi.load()
    for name in OK:
        f = getattr(lib, name)
        if name + "_workspace_size" not in abi.EXPORTS:
            assert f(None, None) == 1
            continue
        assert f(None, None, 0, None) == 1 and getattr(lib, name + "_workspace_size")(None) == 0
        a = raw(abi, name)
        need = abi.ENTRIES[name].workspace_size(a)
        assert need > 256
        assert f(a, None, 0, None) == 3 and f(a, 4096, need - 1, None) == 3 and f(a, 4100, need, None) == 3


def test_empty_problems_are_host_side_no_ops(abi):
    assert call(abi, "gdn_conv_step", N=0) == 0
    assert call(abi, "gdn_ssm_step", N=0) == 0
    assert call(abi, "gdn_ffn_fwd", M=0) == 0
    assert abi.ENTRIES["gdn_conv_bwd"].workspace_size(raw(abi, "gdn_conv_bwd", T=0)) == 256


def test_workspaces_stay_small_beside_the_data(abi):
    """A row of partial sums for each run of tokens: as many as fill the GPU, however long the batch."""
    size = lambda **kw: abi.ENTRIES["gdn_conv_bwd"].workspace_size(raw(abi, "gdn_conv_bwd", B=1, **kw))
    assert size(T=1 << 30, D=64) <= 1 << 24 and size(T=1 << 20, D=4096) <= 1 << 25
    assert size(T=TOP - (1 << 17), D=1) <= 1 << 24
