"""Refusals of the speculative-decoding entry points, without a GPU: every
argument error is found before anything is launched, and a valid call where no
GB300 is present fails loudly."""
import ctypes

import pytest

from tests.test_abi_host import fake, fwlib  # noqa: F401

BF, F32, I32, E4M3 = 0, 1, 2, 3
OK, INVALID, UNSUPPORTED = 0, 1, 2


def ref(t):
    return ctypes.addressof(t) if t is not None else None


def at(shape, dtype, ptr, strides=None):
    return fake(shape, dtype, ptr=ptr, strides=strides)


def tree_args(B=2, T=5, Hq=8, Hkv=2, D=128, P=10, ps=16, width=4, kv=BF):
    return dict(q=fake([B, T, Hq, D], BF), k=fake([P, ps, Hkv, D], kv), v=fake([P, ps, Hkv, D], kv),
                bt=fake([B, width], I32), sl=fake([B], I32), mask=fake([B, T, -(-T // 32)], I32), dl=fake([B], I32),
                scale=0.1, ks=1.0, vs=1.0, out=fake([B, T, Hq, D], BF), lse=fake([B, T, Hq], F32))


def call_tree(fw, a):
    return fw.load_library().fw_paged_decode_tree(
        ref(a["q"]), ref(a["k"]), ref(a["v"]), ref(a["bt"]), ref(a["sl"]), ref(a["mask"]), ref(a["dl"]), a["scale"],
        a["ks"], a["vs"], ref(a["out"]), ref(a["lse"]), None, 0, None)


def setter(name, value):
    return lambda a: a.__setitem__(name, value)


@pytest.mark.parametrize("change,status", [
    (setter("q", None), INVALID),
    (setter("mask", None), INVALID),
    (setter("sl", None), INVALID),
    (setter("out", None), INVALID),
    (setter("q", fake([2, 5, 8, 128], F32)), INVALID),
    (setter("k", fake([10, 16, 2, 128], E4M3)), INVALID),                    # K and V of different types
    (setter("v", fake([10, 16, 2, 64], BF)), UNSUPPORTED),
    (setter("v", fake([9, 16, 2, 128], BF)), INVALID),
    (setter("bt", fake([3, 4], I32)), INVALID),
    (setter("bt", fake([2, 4], I32, strides=[8, 2])), INVALID),
    (setter("bt", fake([2, 4], I32, ptr=0x10002)), INVALID),
    (setter("sl", fake([3], I32)), INVALID),
    (setter("sl", fake([2], I32, strides=[2])), INVALID),
    (setter("dl", fake([3], I32)), INVALID),
    (setter("mask", fake([2, 5, 0], I32)), INVALID),
    (setter("mask", fake([2, 4, 1], I32)), INVALID),
    (setter("mask", fake([2, 5, 1], F32)), INVALID),
    (setter("scale", float("nan")), INVALID),
    (setter("scale", float("inf")), INVALID),
    (setter("ks", 2.0), INVALID),                                            # BF16 caches take no scales
    (setter("out", fake([2, 5, 8, 64], BF)), INVALID),
    (setter("out", fake([2, 5, 8, 128], BF, ptr=0x10008)), INVALID),
    (setter("out", fake([2, 5, 8, 128], BF, strides=[5 * 8 * 132, 8 * 132, 132, 1])), INVALID),
    (setter("lse", fake([2, 5, 7], F32)), INVALID),
    (setter("lse", fake([2, 5, 8], BF)), INVALID),
    (setter("out", fake([2, 5, 8, 128], BF, strides=[0, 1024, 128, 1])), INVALID),         # rows written twice
    (setter("out", fake([2, 5, 8, 128], BF, strides=[5120, 1024, 64, 1])), INVALID),
    (setter("lse", fake([2, 5, 8], F32, strides=[40, 0, 1])), INVALID),
    (setter("q", fake([2, 5, 8, 128], BF, ptr=0x10004)), INVALID),
    (setter("k", fake([10, 16, 2, 128], BF, strides=[16 * 260, 260, 130, 1])), INVALID),
])
def test_tree_decode_refusals(fwlib, change, status):  # noqa: F811
    a = tree_args()
    change(a)
    assert call_tree(fwlib, a) == status, fwlib.load_library().fw_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(T=257), UNSUPPORTED), (dict(T=0), UNSUPPORTED), (dict(B=4097), UNSUPPORTED), (dict(D=64), UNSUPPORTED),
    (dict(D=256, kv=E4M3), UNSUPPORTED), (dict(ps=24), UNSUPPORTED), (dict(Hq=6, Hkv=4), INVALID),
    (dict(P=0), INVALID), (dict(width=0), INVALID),
    (dict(width=1 << 27), UNSUPPORTED),                                     # 2^31 keys
])
def test_tree_decode_sizes(fwlib, kw, status):  # noqa: F811
    assert call_tree(fwlib, tree_args(**kw)) == status, fwlib.load_library().fw_last_error()


@pytest.mark.parametrize("ks,vs", [(0.0, 1.0), (1.0, -1.0), (float("inf"), 1.0), (1.0, float("nan"))])
def test_tree_decode_scales_of_fp8_caches(fwlib, ks, vs):  # noqa: F811
    a = tree_args(kv=E4M3)
    a["ks"], a["vs"] = ks, vs
    assert call_tree(fwlib, a) == INVALID


def call_mask(fw, parents, dl, mask, depths):
    return fw.load_library().fw_tree_mask(ref(parents), ref(dl), ref(mask), ref(depths), None)


def test_tree_mask_refusals(fwlib):  # noqa: F811
    p, d, m, e = fake([2, 40], I32), fake([2], I32), fake([2, 40, 2], I32), fake([2, 40], I32)
    assert call_mask(fwlib, None, d, m, e) == INVALID
    assert call_mask(fwlib, p, d, None, e) == INVALID
    assert call_mask(fwlib, fake([2, 40], F32), d, m, e) == INVALID
    assert call_mask(fwlib, p, fake([3], I32), m, e) == INVALID
    assert call_mask(fwlib, p, d, fake([2, 40, 1], I32), e) == INVALID
    assert call_mask(fwlib, p, d, m, fake([2, 39], I32)) == INVALID
    assert call_mask(fwlib, p, d, fake([2, 40, 2], I32, strides=[160, 4, 2]), e) == INVALID
    p, d, m, e = at([2, 40], I32, 0x10000), at([2], I32, 0x20000), at([2, 40, 2], I32, 0x30000), at([2, 40], I32, 0x40000)
    assert call_mask(fwlib, p, d, at([2, 40, 2], I32, 0x30000, [0, 2, 1]), e) == INVALID
    assert call_mask(fwlib, p, d, m, at([2, 40], I32, 0x40000, [39, 1])) == INVALID
    assert call_mask(fwlib, p, d, m, p) == INVALID
    assert call_mask(fwlib, p, d, at([2, 40, 2], I32, 0x10080), e) == INVALID
    assert call_mask(fwlib, p, d, m, at([2, 40], I32, 0x30004)) == INVALID
    assert call_mask(fwlib, p, d, m, at([2, 40], I32, 0x10000 + 4 * 39, [80, 1])) == INVALID
    assert call_mask(fwlib, fake([2, 257], I32), d, fake([2, 257, 9], I32), None) == UNSUPPORTED
    assert call_mask(fwlib, fake([2, 0], I32), d, fake([2, 0, 0], I32), None) == UNSUPPORTED


def table_args(B=4, width=6, F=50, N=20, L=None):
    return dict(seq=at([B], I32, 0x10000), new=at([B], I32, 0x20000), held=at([B], I32, 0x30000),
                queue=at([F], I32, 0x40000), range=at([2], I32, 0x50000), ps=16, bt=at([B, width], I32, 0x60000),
                slots=at([N] if L is None else [B, L], I32, 0x70000), cu=at([B + 1], I32, 0x80000),
                held_out=at([B], I32, 0x90000), range_out=at([2], I32, 0xa0000))


def call_tables(fw, a):
    return fw.load_library().fw_build_page_tables(
        ref(a["seq"]), ref(a["new"]), ref(a["held"]), ref(a["queue"]), ref(a["range"]), a["ps"], ref(a["bt"]),
        ref(a["slots"]), ref(a["cu"]), ref(a["held_out"]), ref(a["range_out"]), None)


@pytest.mark.parametrize("change", [
    setter("seq", None), setter("new", at([3], I32, 0x20000)), setter("held", at([4], F32, 0x30000)),
    setter("queue", None), setter("range", at([3], I32, 0x50000)), setter("ps", 0), setter("ps", (1 << 20) + 1),
    setter("bt", at([4, 6], I32, 0x60000, [12, 2])), setter("bt", at([5, 6], I32, 0x60000)),
    setter("slots", None), setter("slots", at([4, 5, 1], I32, 0x70000)), setter("slots", at([3, 5], I32, 0x70000)),
    setter("slots", at([4, 5], I32, 0x70000, [6, 1])), setter("slots", at([20], I32, 0x70000, [2])),
    setter("cu", at([4], I32, 0x80000)), setter("held_out", None), setter("range_out", at([1], I32, 0xa0000)),
    setter("slots", at([20], I32, 0x10000)),                                 # over seq_lens
    setter("held_out", at([4], I32, 0x20004)),                               # over new_lens
    setter("held_out", at([4], I32, 0x30004)),                               # held, but for one entry
    setter("range_out", at([2], I32, 0x50004)),
    setter("bt", at([4, 6], I32, 0x60000, [0, 1])), setter("bt", at([4, 6], I32, 0x60000, [5, 1])),
    setter("cu", at([5], I32, 0x70000)),                                     # over the slots
    setter("queue", at([50], I32, 0x60010)),                                 # over the table
])
def test_page_table_refusals(fwlib, change):  # noqa: F811
    a = table_args()
    change(a)
    assert call_tables(fwlib, a) == INVALID, fwlib.load_library().fw_last_error()


def test_page_table_sizes(fwlib):  # noqa: F811
    a = table_args()
    a["queue"] = at([0], I32, 0x40000)
    assert call_tables(fwlib, a) == UNSUPPORTED
    a = table_args()
    a["slots"] = at([2 ** 30 + 1], I32, 0x70000)
    assert call_tables(fwlib, a) == UNSUPPORTED
    B = 8193
    a = table_args(B=B, width=0, N=1)
    for i, k in enumerate(("seq", "new", "held", "held_out", "slots", "cu")):
        a[k].data = 0x100000 * (i + 1)
    assert call_tables(fwlib, a) == UNSUPPORTED


def commit_args(B=3, A=4, P=12, ps=16, Hkv=2, D=128, width=5, kv=BF):
    size = P * ps * Hkv * D * 2
    return dict(path=fake([B, A], I32, 0x1000), pl=fake([B], I32, 0x2000), bl=fake([B], I32, 0x3000),
                bt=fake([B, width], I32, 0x4000), layers=3, k=fake([P, ps, Hkv, D], kv, 0x100000),
                v=fake([P, ps, Hkv, D], kv, 0x100000 + size), new=fake([B], I32, 0x5000))


def call_commit(fw, a):
    return fw.load_library().fw_kv_commit(ref(a["path"]), ref(a["pl"]), ref(a["bl"]), ref(a["bt"]), a["layers"],
                                          ref(a["k"]), ref(a["v"]), ref(a["new"]), None)


@pytest.mark.parametrize("change,status", [
    (setter("path", None), INVALID), (setter("path", fake([3, 4], I32, strides=[8, 2])), INVALID),
    (setter("pl", fake([2], I32)), INVALID), (setter("bl", None), INVALID), (setter("bt", fake([2, 5], I32)), INVALID),
    (setter("layers", 0), INVALID), (setter("layers", 5), INVALID), (setter("k", None), INVALID),
    (setter("k", fake([12, 16, 2, 128], F32, 0x100000)), INVALID),
    (setter("v", fake([12, 16, 2, 128], E4M3, 0x900000)), INVALID),
    (setter("v", fake([12, 16, 1, 128], BF, 0x900000)), INVALID),
    (setter("v", fake([12, 16, 2, 128], BF, 0x100000)), INVALID),            # the keys themselves
    (setter("v", fake([12, 16, 2, 64], BF, 0x100080, [16 * 256, 256, 128, 1])), INVALID),   # a view of the keys
    (setter("v", fake([12, 16, 2, 128], BF, 0x900008)), INVALID),
    (setter("k", fake([12, 16, 2, 128], BF, 0x900000, [0, 256, 128, 1])), INVALID),         # a page written many times
    (setter("path", fake([3, 257], I32, 0x1000)), UNSUPPORTED),
    (setter("new", fake([3], I32, 0x3004)), INVALID),                        # over base_lens
])
def test_commit_refusals(fwlib, change, status):  # noqa: F811
    a = commit_args()
    change(a)
    assert call_commit(fwlib, a) == status, fwlib.load_library().fw_last_error()


def test_commit_row_sizes(fwlib):  # noqa: F811
    a = commit_args(D=12)
    assert call_commit(fwlib, a) == UNSUPPORTED
    a = commit_args(D=8, kv=E4M3)
    assert call_commit(fwlib, a) == UNSUPPORTED


def test_valid_calls_without_a_gpu_fail_loudly(fwlib):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    n = fwlib.launch_count()
    half = commit_args()
    page = 16 * 2 * 128                                       # K and V the halves of every page of one buffer
    half["k"] = fake([12, 16, 2, 128], BF, 0x100000, [2 * page, 256, 128, 1])
    half["v"] = fake([12, 16, 2, 128], BF, 0x100000 + 2 * page, [2 * page, 256, 128, 1])
    same = table_args()
    same["held_out"], same["range_out"] = same["held"], same["range"]        # may be their inputs
    for rc in (call_tree(fwlib, tree_args()), call_tree(fwlib, tree_args(kv=E4M3)),
               call_mask(fwlib, fake([2, 40], I32), None, fake([2, 40, 2], I32, 0x90000), None),
               call_mask(fwlib, at([2, 40], I32, 0x10000, [80, 1]), None, fake([2, 40, 2], I32, 0x90000),
                         at([2, 40], I32, 0x10000 + 160, [80, 1])),       # columns of one buffer
               call_tables(fwlib, table_args()), call_tables(fwlib, table_args(L=5)), call_tables(fwlib, same),
               call_commit(fwlib, commit_args()), call_commit(fwlib, half)):
        assert rc in (2, 4), fwlib.load_library().fw_last_error()
    assert fwlib.launch_count() == n


def test_cpu_tensors_are_refused(fwlib):  # noqa: F811
    import torch
    z = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fwlib.tree_mask(z)
    with pytest.raises(ValueError, match="CUDA"):
        fwlib.kv_commit(z, z[:, 0], z[:, 0], z, torch.zeros(1, 1, 1, 8), None)
