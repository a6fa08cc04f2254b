"""A step's new states over the old ones, or apart from them, but not half over them: refused on the host."""
import pytest

import test_abi_block
import test_abi_layer
from test_abi_layer import abi  # noqa: F401  (a fixture)

OK = {**test_abi_block.OK, **test_abi_layer.OK}
BYTES = {("gdn_conv_step", 0): 2 * 3 * 64 * 4, ("gdn_conv_step", 1): 2 * 3 * 64 * 2, ("gdn_ssm_step", 0): 2 * 64 * 16 * 4,
         ("gdn_ssm_step", 1): 2 * 64 * 16 * 4, ("gdn_linrec_step", 1): 2 * 64 * 4}


@pytest.mark.parametrize("name,dtype", list(BYTES))
def test_states_that_overlap(abi, name, dtype):
    size, at = BYTES[name, dtype], 1 << 20
    for state, out in ((at, at + 16), (at + 16, at), (at, at + size - 16), (at + size - 16, at)):
        a = getattr(abi, name + "_args")()
        for k, v in {**OK[name], "dtype": dtype, "state": state, "out_state": out}.items():
            setattr(a, k, v)
        assert getattr(abi.load(), name)(bytes(a), None) == 1
        assert "overlaps" in abi._abi.gdn_last_error()
