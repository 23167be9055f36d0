"""Tree decode: what is written may lie over nothing else of the call; views of one
buffer that share no element are fine.  A refused call launches nothing."""
import pytest
import torch

from oracle import spec
from tests.gpu_common import built_library
from tests.test_tree_decode_gpu import check, make, on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    return built_library()


def test_outputs_over_anything_else_are_refused(fw):
    x = make(2, 6, 8, 2, 128, 16, [100, 60], [6, 4], "tree", seed=91)
    g = on_gpu(x)
    n = fw.paged_decode_tree_workspace_size(128)
    ws = torch.empty(n + 4096, dtype=torch.uint8, device="cuda")
    q, rows = g["q"], 2 * 6 * 8
    lse = torch.empty(2, 6, 8, device="cuda")
    out = torch.empty_like(q)
    flat = lambda t, dt, m: t.view(torch.uint8).view(-1)[:m].view(dt)
    before = fw.launch_count()
    cases = {
        "q": dict(out=q),
        "k_cache": dict(out=flat(g["k_cache"], torch.bfloat16, 2 * rows * 128).view(q.shape)),
        "v_cache": dict(lse=flat(g["v_cache"], torch.float32, 4 * rows).view(2, 6, 8)),
        "lse": dict(out=out, lse=flat(out, torch.float32, 4 * rows).view(2, 6, 8)),
        "overlaps q": dict(lse=flat(q, torch.float32, 4 * rows).view(2, 6, 8)),
        "the workspace overlaps out": dict(out=ws[:2 * rows * 128].view(torch.bfloat16).view(q.shape), workspace=ws),
        "the workspace overlaps lse": dict(lse=ws[n - 256:][:4 * rows].view(torch.float32).view(2, 6, 8), workspace=ws),
    }
    for name, kw in cases.items():
        with pytest.raises(fw.FwError, match=name):
            fw.paged_decode_tree(**g, **kw)
    big = torch.zeros(2 * 6 * 8 * 128 // 2, dtype=torch.int32, device="cuda")      # masks and lengths inside out
    inside = dict(g, tree_mask=big[:12].view(2, 6, 1))
    inside["tree_mask"].copy_(g["tree_mask"])
    with pytest.raises(fw.FwError, match="tree_mask"):
        fw.paged_decode_tree(**inside, out=big.view(torch.bfloat16).view(q.shape))
    inside = dict(g, seq_lens=big[:2])
    with pytest.raises(fw.FwError, match="seq_lens"):
        fw.paged_decode_tree(**inside, out=big.view(torch.bfloat16).view(q.shape))
    assert fw.launch_count() == before
    torch.cuda.synchronize()
    assert fw.device_status() == 0


def test_columns_of_one_buffer(fw):
    """Queries and outputs as columns of one buffer, which share no element."""
    x = make(2, 6, 8, 2, 128, 16, [100, 60], [6, 4], "tree", seed=93)
    g = on_gpu(x)
    buf = torch.zeros(2, 6, 16, 128, dtype=torch.bfloat16, device="cuda")
    buf[:, :, :8] = g["q"]
    g["q"] = buf[:, :, :8]
    out, lse = fw.paged_decode_tree(**g, out=buf[:, :, 8:])
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    check(out, lse, spec.tree_attention(**x), 128, "columns")
    assert torch.equal(buf[:, :, :8].cpu(), x["q"])
