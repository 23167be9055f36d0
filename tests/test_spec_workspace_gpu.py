"""A caller's workspace of no bytes is too small, not absent."""
import pytest
import torch

from tests.gpu_common import built_library
from tests.test_tree_decode_gpu import make, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float32])
def test_an_empty_workspace_is_refused(dtype):
    fw = built_library()
    x = on_gpu(make(1, 4, 8, 2, 128, 16, [100], None, "tree", seed=95))
    before = fw.launch_count()
    with pytest.raises(fw.FwError, match="workspace holds 0 bytes"):
        fw.paged_decode_tree(**x, workspace=torch.empty(0, dtype=dtype, device="cuda"))
    assert fw.launch_count() == before
