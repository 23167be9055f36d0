"""Verification of drafts: rows that are no probabilities, at nodes that the path goes
through."""
import pytest
import torch

from tests.gpu_common import built_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    return built_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [8, 40000])
def test_a_row_of_four_and_more_is_told_where_a_draft_is_rejected(fw, V, draft):
    """Draft 1 is rejected at a row of ones, draft 2 accepted there: the path ends at a row
    that is one, and the call still tells."""
    target = torch.zeros(1, 3, V, device="cuda")
    target[0, 0] = 1.0
    target[0, 0, 5] = 0.0
    target[0, 1:, 3] = 1.0
    q = torch.zeros_like(target)
    q[:, :, 5], q[:, :, 6] = 0.5, 0.125
    args = (i32([[0, 5, 6]]), i32([[-1, 0, 0]]), target, torch.tensor([[0.0, 0.9, 0.1, 0.5]], device="cuda"))
    fw.device_status()
    path, n, nxt = fw.verify_drafts(*args, draft_probs=q if draft else None)
    assert (path.tolist(), n.tolist(), nxt.tolist()) == ([[0, 2, -1]], [2], [3])
    assert fw.device_status() == 1
    target[0, 0, :5] = target[0, 0, 7:] = 0.0             # the one at 6 is left: fine
    path, n, nxt = fw.verify_drafts(*args, draft_probs=q if draft else None)
    assert (path.tolist(), n.tolist(), nxt.tolist()) == ([[0, 2, -1]], [2], [3])
    assert fw.device_status() == 0


def test_a_path_of_another_width_than_max_path_is_refused(fw):
    """How many drafts may be accepted is said once: by the width of a given path."""
    probs = torch.full((1, 3, 4), 0.25, device="cuda")
    args = (i32([[0, 1, 2]]), i32([[-1, 0, 1]]), probs, torch.zeros(1, 4, device="cuda"))
    path = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    before = fw.launch_count()
    for given, most in ((path, 1), (path, 4), (path[:, :2], 3), (path[0], 3)):
        with pytest.raises(ValueError, match="max_path"):
            fw.verify_drafts(*args, max_path=most, path=given)
    assert fw.launch_count() == before
    for given, most in ((path, 3), (path, None), (path[:, :1], 1), (None, 2)):
        got, n, _ = fw.verify_drafts(*args, max_path=most, path=given)
        want = 3 if given is path else 1 if given is not None else 2
        assert got.shape == (1, want) and n.tolist() == [want]
