"""Refusals of the speculative entry points at their limits, without a GPU: sizes at
which an index would leave 32 bits, a commit whose caches hold its own vectors."""
import pytest

from tests.test_abi_host import fake, fwlib  # noqa: F401
from tests.test_spec_host import BF, F32, I32, INVALID, UNSUPPORTED, call_commit, call_tree, commit_args, tree_args


@pytest.mark.parametrize("D,Hq,fits", [(128, 1 << 27, False), (256, 1 << 26, False), (128, (1 << 27) - 8, True),
                                       (256, (1 << 26) - 8, True)])
def test_units_of_a_padding_row(fwlib, D, Hq, fits):  # noqa: F811
    a = tree_args(B=1, T=1, Hq=Hq, Hkv=1, D=D)
    a["out"] = fake([1, 1, Hq, D], BF, ptr=1 << 40)
    a["lse"] = fake([1, 1, Hq], F32, ptr=1 << 41)
    rc = call_tree(fwlib, a)
    message = fwlib.load_library().fw_last_error().decode()
    assert (rc == UNSUPPORTED and "heads" in message) != fits, (rc, message)


@pytest.mark.parametrize("name,shape", [("path", [3, 4]), ("pl", [3]), ("bl", [3]), ("bt", [3, 5]), ("new", [3])])
@pytest.mark.parametrize("cache", ["k", "v"])
def test_commit_vectors_inside_a_cache(fwlib, name, shape, cache):  # noqa: F811
    a = commit_args()
    assert call_commit(fwlib, a) != INVALID
    a[name] = fake(shape, I32, a[cache].data + 4096)
    assert call_commit(fwlib, a) == INVALID and b"cache overlaps" in fwlib.load_library().fw_last_error()
    page = 16 * 2 * 128                                       # a page's metadata behind it, in one buffer
    for i, c in enumerate("kv"):
        a[c] = fake([12, 16, 2, 128], BF, 0x100000 + 2 * page * i, [2 * page + 256, 256, 128, 1])
    a[name] = fake(shape, I32, 0x100000 + 4 * page)
    assert call_commit(fwlib, a) != INVALID, fwlib.load_library().fw_last_error()


def test_a_stream_without_tensors(fwlib):  # noqa: F811
    """The error names the argument, with a stream as without one."""
    for stream in (None, object()):
        with pytest.raises(TypeError, match="parents is required"):
            fwlib.tree_mask(None, stream=stream)
        with pytest.raises(TypeError, match="q must be a torch.Tensor"):
            fwlib.paged_decode_tree([1], None, None, None, None, None, 1.0, stream=stream)
