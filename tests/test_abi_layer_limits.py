"""Host-side refusals of the microscaled operators: sizes near 2^31, and bad arguments of the linear
entry before it launches anything (here, without a GPU, anything that it would launch is another error)."""
import pytest

from test_abi_layer import abi, call, raw  # noqa: F401  (a fixture)

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("bad,rc,msg", [
    (dict(w=None), 1, "required"), (dict(w_scales=None), 1, "required"), (dict(c=None), 1, "required"),
    (dict(w=4100), 1, "aligned"), (dict(w_scales=4104), 1, "aligned"), (dict(c=4098), 1, "aligned"),
    (dict(x=4098), 1, "aligned"), (dict(N=-1), 1, "bad sizes"), (dict(out_dtype=7), 2, "out_dtype"),
    (dict(format=2), 2, "format"), (dict(dtype=5), 2, "dtype"), (dict(out_dtype=7, M=1000), 2, "out_dtype"),
    (dict(c=4098, M=1000), 1, "aligned"),
])
def test_linear_checks_everything_before_it_launches(abi, bad, rc, msg):
    assert call(abi, "gdn_mx_linear", **bad) == rc
    assert msg in abi._abi.gdn_last_error()


def test_linear_of_no_rows_or_columns_launches_nothing(abi):
    assert call(abi, "gdn_mx_linear", M=0) == 0
    assert call(abi, "gdn_mx_linear", N=0) == 0


@pytest.mark.parametrize("name,big", [
    ("gdn_mx_quantize", dict(K=2 ** 31 - 32)), ("gdn_mx_dequantize", dict(K=2 ** 31 - 32)),
    ("gdn_mx_matmul", dict(M=TOP, N=1, K=32)), ("gdn_mx_matmul", dict(M=1, N=TOP - 100, K=32)),
    ("gdn_mx_matmul", dict(K=2 ** 31 - 32)),
    ("gdn_mx_linear", dict(M=TOP, N=1, K=32)), ("gdn_mx_linear", dict(M=1, N=TOP - 100, K=32)),
    ("gdn_mx_linear", dict(K=2 ** 31 - 64)),
])
def test_sizes_whose_arithmetic_would_overflow_are_refused(abi, name, big):
    assert call(abi, name, **big) == 1
    assert "too large" in abi._abi.gdn_last_error()


def test_no_workspace_is_named_for_them(abi):
    assert abi.load().gdn_mx_linear_workspace_size(raw(abi, "gdn_mx_linear", M=TOP)) == 0
    assert "too large" in abi._abi.gdn_last_error()


def test_the_norms_backward_of_very_many_rows_asks_for_as_many_sums_as_of_fewer(abi):
    """A row of partial sums of d(weight) for each CTA: as many as the GPU holds, not as many as an int
    that overflowed says."""
    size = lambda rows: abi.ENTRIES["gdn_rms_norm_bwd"].workspace_size(raw(abi, "gdn_rms_norm_bwd", rows=rows, D=1))
    assert size(TOP) == size(2 ** 30) > 1024
