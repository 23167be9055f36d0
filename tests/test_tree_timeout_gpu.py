"""The bounded device waits of the tree decode kernels: a wait that runs out
reports FW_ERR_DEVICE_TIMEOUT, the warps that share barriers leave together, and
the library stays usable.

FW_OPT_TEST_STALL makes the warp that copies keys and values wait, before it
copies any, on a barrier that nothing completes.  No product begins without a
key tile, so when that wait runs out no copy but the queries' own (which land)
and no MMA is in flight; the other warps go over the units at hand without data
and meet at the end.
"""
import pytest
import torch

from tests.gpu_common import built_library
from tests.test_tree_decode_gpu import make, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctas", [0, 3])           # a unit or a cut one to a CTA, and many
@pytest.mark.parametrize("T,Hq,Hkv", [(9, 8, 2), (40, 16, 4)])
@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
def test_a_wait_that_runs_out(D, kv8, T, Hq, Hkv, ctas):
    fw = built_library()
    x = on_gpu(make(4, T, Hq, Hkv, D, 32, [900, T, 300, 77], None, "tree", kv8=kv8, seed=81))
    assert fw.device_status() == 0
    fw.set_option(fw.FW_OPT_MAX_CTAS, ctas)
    try:
        alone = fw.paged_decode_tree(**x)
        torch.cuda.synchronize()
        assert fw.device_status() == 0
        fw.set_option(fw.FW_OPT_WAIT_TIMEOUT_MS, 1)    # the shortest limit
        fw.set_option(fw.FW_OPT_TEST_STALL, 1)
        fw.paged_decode_tree(**x)                      # the call itself is accepted
        torch.cuda.synchronize()
        assert fw.device_status() == fw.FW_ERR_DEVICE_TIMEOUT
        fw.set_option(fw.FW_OPT_TEST_STALL, 0)
        fw.set_option(fw.FW_OPT_WAIT_TIMEOUT_MS, 2000)
        assert fw.device_status() == 0                 # reading the word cleared it
        for _ in range(2):
            again = fw.paged_decode_tree(**x)
            torch.cuda.synchronize()
            assert fw.device_status() == 0
            assert torch.equal(again[0], alone[0]) and torch.equal(again[1], alone[1])
    finally:
        fw.set_option(fw.FW_OPT_TEST_STALL, 0)
        fw.set_option(fw.FW_OPT_WAIT_TIMEOUT_MS, 2000)
        fw.set_option(fw.FW_OPT_MAX_CTAS, 0)
