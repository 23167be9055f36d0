"""Sizes at which an index of the speculative entry points would leave 32 bits are
refused, those below are not, without a GPU."""
import pytest

from tests.test_abi_host import fake, fwlib  # noqa: F401
from tests.test_spec_host import BF, F32, UNSUPPORTED, call_tree, tree_args


@pytest.mark.parametrize("D,Hq,fits", [(128, 1 << 27, False), (256, 1 << 26, False), (128, (1 << 27) - 8, True),
                                       (256, (1 << 26) - 8, True)])
def test_units_of_a_padding_row(fwlib, D, Hq, fits):  # noqa: F811
    a = tree_args(B=1, T=1, Hq=Hq, Hkv=1, D=D)
    a["out"] = fake([1, 1, Hq, D], BF, ptr=1 << 40)
    a["lse"] = fake([1, 1, Hq], F32, ptr=1 << 41)
    rc = call_tree(fwlib, a)
    message = fwlib.load_library().fw_last_error().decode()
    assert (rc == UNSUPPORTED and "heads" in message) != fits, (rc, message)
