"""Refusals of the entry points around a step's attention, without a GPU: every argument
error is found before anything is launched, and a valid call where no GB300 is present
fails loudly."""
import ctypes

import pytest

from tests.test_abi_host import fake, fwlib  # noqa: F401
from tests.test_spec_host import ref

BF, F32, I32, E4M3 = 0, 1, 2, 3
OK, INVALID, UNSUPPORTED = 0, 1, 2


def setter(name, value):
    return lambda a: a.__setitem__(name, value)


def at(shape, dtype, ptr, strides=None):
    return fake(shape, dtype, ptr=ptr, strides=strides)


def says(fw):
    return fw.load_library().fw_last_error().decode()


# ------------------------------------------------------------- chunk attention

def prefill_args(N=30, B=3, Hq=8, Hkv=2, D=128, P=10, ps=16, width=4, kv=BF):
    return dict(q=at([N, Hq, D], BF, 0x100000), k=at([P, ps, Hkv, D], kv, 0x10000000), v=at([P, ps, Hkv, D], kv, 0x20000000),
                bt=at([B, width], I32, 0x30000000), cu=at([B + 1], I32, 0x31000000), sl=at([B], I32, 0x32000000), scale=0.1,
                ks=1.0, vs=1.0, causal=1, window=-1, out=at([N, Hq, D], BF, 0x40000000), lse=at([N, Hq], F32, 0x50000000),
                ws=None, bytes=0)


def call_prefill(fw, a):
    return fw.load_library().fw_paged_prefill(
        ref(a["q"]), ref(a["k"]), ref(a["v"]), ref(a["bt"]), ref(a["cu"]), ref(a["sl"]), a["scale"], a["ks"], a["vs"],
        a["causal"], a["window"], ref(a["out"]), ref(a["lse"]), a["ws"], a["bytes"], None)


@pytest.mark.parametrize("change,status", [
    *[(setter(n, None), INVALID) for n in ("q", "k", "v", "bt", "cu", "sl", "out")],
    (setter("q", fake([30, 8, 128], F32)), INVALID),
    (setter("q", fake([30, 2, 4, 128], BF)), INVALID),
    (setter("k", fake([10, 16, 2, 128], E4M3)), INVALID),                    # K and V of different types
    (setter("k", fake([10, 16, 2, 128], F32)), INVALID),
    (setter("k", fake([10, 16, 2, 256], BF)), INVALID),
    (setter("v", fake([10, 16, 2, 64], BF)), UNSUPPORTED),
    (setter("v", fake([9, 16, 2, 128], BF)), INVALID),
    (setter("bt", fake([3, 4], F32)), INVALID),
    (setter("bt", fake([3, 4], I32, strides=[8, 2])), INVALID),
    (setter("bt", fake([3, 4], I32, ptr=0x10002)), INVALID),
    (setter("cu", fake([3], I32)), INVALID),
    (setter("cu", fake([4], I32, strides=[2])), INVALID),
    (setter("sl", fake([4], I32)), INVALID),
    (setter("scale", float("nan")), INVALID),
    (setter("scale", float("inf")), INVALID),
    (setter("ks", 2.0), INVALID),                                            # BF16 caches take no scales
    (setter("window", -2), INVALID),
    (setter("out", fake([30, 8, 64], BF)), INVALID),
    (setter("out", fake([29, 8, 128], BF)), INVALID),
    (setter("out", fake([30, 8, 128], BF, ptr=0x10008)), INVALID),
    (setter("out", fake([30, 8, 128], BF, strides=[0, 128, 1])), INVALID),         # rows written twice
    (setter("out", fake([30, 8, 128], BF, strides=[1024, 64, 1])), INVALID),
    (setter("out", fake([30, 8, 128], BF, strides=[1056, 132, 1])), INVALID),
    (setter("lse", fake([30, 7], F32)), INVALID),
    (setter("lse", fake([30, 8], BF)), INVALID),
    (setter("lse", fake([30, 8], F32, strides=[0, 1])), INVALID),
    (setter("q", fake([30, 8, 128], BF, ptr=0x10004)), INVALID),
    (setter("k", fake([10, 16, 2, 128], BF, strides=[16 * 260, 260, 130, 1])), INVALID),
])
def test_prefill_refusals(fwlib, change, status):  # noqa: F811
    a = prefill_args()
    change(a)
    assert call_prefill(fwlib, a) == status, says(fwlib)


@pytest.mark.parametrize("kw,status", [
    (dict(B=4097), UNSUPPORTED), (dict(D=64), UNSUPPORTED), (dict(D=256, kv=E4M3), UNSUPPORTED), (dict(ps=24), UNSUPPORTED),
    (dict(ps=192), UNSUPPORTED), (dict(Hq=6, Hkv=4), INVALID), (dict(Hq=0), INVALID), (dict(P=0), INVALID), (dict(width=0), INVALID),
    (dict(width=1 << 27), UNSUPPORTED),                                     # 2^31 keys
    (dict(N=1 << 28, Hq=8), UNSUPPORTED),                                   # 2^31 rows
])
def test_prefill_sizes(fwlib, kw, status):  # noqa: F811
    assert call_prefill(fwlib, prefill_args(**kw)) == status, says(fwlib)


@pytest.mark.parametrize("ks,vs", [(0.0, 1.0), (1.0, -1.0), (float("inf"), 1.0), (1.0, float("nan"))])
def test_prefill_scales_of_fp8_caches(fwlib, ks, vs):  # noqa: F811
    a = prefill_args(kv=E4M3)
    a["ks"], a["vs"] = ks, vs
    assert call_prefill(fwlib, a) == INVALID


def test_prefill_of_nothing_is_fine(fwlib):  # noqa: F811
    for kw in (dict(N=0), dict(B=0)):
        assert call_prefill(fwlib, prefill_args(**kw)) == OK, says(fwlib)


def test_prefill_workspace_size_refuses_other_dims(fwlib):  # noqa: F811
    lib, n = fwlib.load_library(), ctypes.c_size_t(0)
    assert lib.fw_paged_prefill_workspace_size(64, ctypes.byref(n)) == UNSUPPORTED
    assert lib.fw_paged_prefill_workspace_size(128, None) == INVALID


# ------------------------------------------------------------ norm and rotation

def rope_args(N=5, Hq=8, Hkv=2, D=128, F=64, axes=0, kv=BF, P=4, ps=16):
    return dict(q=at([N, Hq, D], BF, 0x100000), k=at([N, Hkv, D], BF, 0x200000), v=at([N, Hkv, D], BF, 0x300000),
                qw=at([D], BF, 0x400000), kw=at([D], F32, 0x410000), eps=1e-6, freq=at([F], F32, 0x420000),
                pos=at([axes, N] if axes else [N], I32, 0x430000), amap=at([F], I32, 0x440000) if axes > 1 else None, inter=0,
                slots=at([N], I32, 0x450000), base=0, qo=at([N, Hq, D], BF, 0x500000), ko=at([N, Hkv, D], BF, 0x600000),
                kc=at([P, ps, Hkv, D], kv, 0x1000000), vc=at([P, ps, Hkv, D], kv, 0x2000000), ks=1.0, vs=1.0)


def call_rope(fw, a, append):
    lib = fw.load_library()
    if append:
        return lib.fw_qk_norm_rope_append(ref(a["q"]), ref(a["k"]), ref(a["v"]), ref(a["qw"]), ref(a["kw"]), a["eps"],
                                          ref(a["freq"]), ref(a["pos"]), ref(a["amap"]), a["inter"], ref(a["slots"]), a["base"],
                                          ref(a["qo"]), ref(a["kc"]), ref(a["vc"]), a["ks"], a["vs"], None)
    return lib.fw_qk_norm_rope(ref(a["q"]), ref(a["k"]), ref(a["qw"]), ref(a["kw"]), a["eps"], ref(a["freq"]), ref(a["pos"]),
                               ref(a["amap"]), a["inter"], ref(a["qo"]), ref(a["ko"]), None)


ROPE = [
    *[(setter(n, None), INVALID) for n in ("q", "k", "freq", "pos", "qo")],
    (setter("q", fake([5, 8, 128], F32)), INVALID),
    (setter("k", fake([4, 2, 128], BF)), INVALID),
    (setter("k", fake([5, 2, 64], BF)), INVALID),
    (setter("k", fake([5, 0, 128], BF)), INVALID),
    (setter("qw", fake([64], BF)), INVALID),
    (setter("kw", fake([128], I32)), INVALID),
    (setter("qw", fake([128], BF, strides=[2])), INVALID),
    (setter("kw", fake([128], F32, ptr=0x10002)), INVALID),
    (setter("eps", float("nan")), INVALID),
    (setter("eps", -1.0), INVALID),
    (setter("freq", fake([65], F32)), UNSUPPORTED),
    (setter("freq", fake([68], F32)), UNSUPPORTED),                          # more than the head
    (setter("freq", fake([0], F32)), UNSUPPORTED),
    (setter("freq", fake([64], BF)), INVALID),
    (setter("pos", fake([4], I32)), INVALID),
    (setter("pos", fake([1, 1, 5], I32)), INVALID),
    (setter("pos", fake([5], F32)), INVALID),
    (setter("pos", fake([2, 5], I32)), INVALID),                             # several axes and no map
    (setter("amap", fake([32], I32)), INVALID),
    (setter("qo", fake([5, 8, 64], BF)), INVALID),
    (setter("qo", fake([5, 8, 128], BF, strides=[0, 128, 1])), INVALID),
    (setter("q", fake([5, 8, 128], BF, ptr=0x100008)), INVALID),
    (setter("q", fake([5, 8, 128], BF, strides=[1056, 132, 1])), INVALID),
    (setter("qo", fake([5, 8, 128], BF, ptr=0x100100)), INVALID),            # over q, but not q
    (setter("qo", fake([5, 8, 128], BF, ptr=0x200000)), INVALID),            # over k
    (setter("qo", fake([5, 8, 128], BF, ptr=0x420000)), INVALID),            # over the frequencies
]


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("change,status", ROPE)
def test_norm_rope_refusals(fwlib, change, status, append):  # noqa: F811
    a = rope_args()
    change(a)
    assert call_rope(fwlib, a, append) == status, says(fwlib)


@pytest.mark.parametrize("change,status", [
    (setter("ko", None), INVALID), (setter("ko", fake([5, 3, 128], BF)), INVALID),
    (setter("ko", fake([5, 2, 128], BF, ptr=0x500000)), INVALID),            # over q_out
])
def test_norm_rope_out_refusals(fwlib, change, status):  # noqa: F811
    a = rope_args()
    change(a)
    assert call_rope(fwlib, a, False) == status, says(fwlib)


@pytest.mark.parametrize("change,status", [
    (setter("kc", None), INVALID), (setter("vc", None), INVALID), (setter("v", None), INVALID), (setter("slots", None), INVALID),
    (setter("slots", fake([4], I32)), INVALID), (setter("slots", fake([5], I32, strides=[2])), INVALID),
    (setter("slots", fake([5], I32, ptr=0x450002)), INVALID),
    (setter("kc", fake([4, 16, 2, 128], E4M3)), INVALID), (setter("kc", fake([4, 16, 3, 128], BF)), INVALID),
    (setter("kc", fake([0, 16, 2, 128], BF)), INVALID), (setter("base", -1), INVALID), (setter("base", 64), INVALID),
    (setter("ks", 0.5), INVALID), (setter("kc", fake([4, 16, 2, 128], BF, ptr=0x2000000)), INVALID),     # K over V
    (setter("kc", fake([4, 16, 2, 128], BF, ptr=0x100000)), INVALID),        # a cache over q
    (setter("kc", fake([4, 16, 2, 128], BF, ptr=0x200000)), INVALID),        # over k: not in place here
    (setter("vc", fake([4, 16, 2, 128], BF, strides=[0, 256, 128, 1])), INVALID),
])
def test_norm_rope_append_refusals(fwlib, change, status):  # noqa: F811
    a = rope_args()
    change(a)
    assert call_rope(fwlib, a, True) == status, says(fwlib)


@pytest.mark.parametrize("kw,status", [(dict(D=96, F=16), UNSUPPORTED), (dict(D=512, F=64), UNSUPPORTED),
                                       (dict(axes=65), UNSUPPORTED), (dict(N=0), OK)])
def test_norm_rope_sizes(fwlib, kw, status):  # noqa: F811
    for append in (False, True):
        assert call_rope(fwlib, rope_args(**kw), append) == status, says(fwlib)


# ------------------------------------------------------------------ verification

def verify_args(B=2, T=4, V=100, R=None, A=4):
    R = T if R is None else R
    return dict(tok=at([B, T], I32, 0x100000), par=at([B, T], I32, 0x110000), dl=at([B], I32, 0x120000),
                tp=at([B, R, V], F32, 0x1000000), dp=at([B, R, V], F32, 0x2000000), u=at([B, T + 1], F32, 0x130000),
                path=at([B, A], I32, 0x140000), pl=at([B], I32, 0x150000), nt=at([B], I32, 0x160000))


def call_verify(fw, a):
    return fw.load_library().fw_verify_drafts(*(ref(a[n]) for n in ("tok", "par", "dl", "tp", "dp", "u", "path", "pl", "nt")), None)


@pytest.mark.parametrize("change,status", [
    *[(setter(n, None), INVALID) for n in ("tok", "par", "tp", "u", "path", "pl", "nt")],
    (setter("tok", fake([2, 4], F32)), INVALID), (setter("par", fake([2, 5], I32)), INVALID),
    (setter("tok", fake([2, 4], I32, strides=[8, 2])), INVALID), (setter("dl", fake([3], I32)), INVALID),
    (setter("tp", fake([2, 4, 100], BF)), INVALID), (setter("tp", fake([2, 3, 100], F32)), INVALID),
    (setter("tp", fake([3, 4, 100], F32)), INVALID), (setter("dp", fake([2, 5, 100], F32)), INVALID),
    (setter("dp", fake([2, 4, 101], F32)), INVALID), (setter("u", fake([2, 4], F32)), INVALID),
    (setter("tp", fake([2, 4, 100], F32, strides=[800, 200, 2])), INVALID),
    (setter("tp", fake([2, 4, 100], F32, ptr=0x10002)), INVALID),
    (setter("path", fake([2, 0], I32)), INVALID), (setter("path", fake([2, 257], I32)), INVALID),
    (setter("path", fake([2, 4], I32, strides=[0, 1])), INVALID), (setter("pl", fake([3], I32)), INVALID),
    (setter("pl", fake([2], I32, ptr=0x160000)), INVALID),                   # over next_tokens
    (setter("nt", fake([2], I32, ptr=0x100000)), INVALID),                   # over the tokens
    (setter("path", fake([2, 4], I32, ptr=0x1000000)), INVALID),             # over the probabilities
])
def test_verify_refusals(fwlib, change, status):  # noqa: F811
    a = verify_args()
    change(a)
    assert call_verify(fwlib, a) == status, says(fwlib)


@pytest.mark.parametrize("kw,status", [(dict(T=257, A=4), UNSUPPORTED), (dict(T=0), UNSUPPORTED), (dict(V=0), UNSUPPORTED),
                                       (dict(V=(1 << 24) + 1), UNSUPPORTED), (dict(B=0), OK), (dict(R=6), INVALID)])
def test_verify_sizes(fwlib, kw, status):  # noqa: F811
    assert call_verify(fwlib, verify_args(**kw)) == status, says(fwlib)


def test_valid_calls_without_a_gpu_fail_loudly(fwlib):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert call_prefill(fwlib, prefill_args()) not in (OK, INVALID)
    assert call_rope(fwlib, rope_args(), False) not in (OK, INVALID)
    assert call_rope(fwlib, rope_args(kv=E4M3), True) not in (OK, INVALID)
    assert call_verify(fwlib, verify_args()) not in (OK, INVALID)


def test_python_entry_points_refuse_what_is_no_gpu_tensor(fwlib):  # noqa: F811
    import torch
    t = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        fwlib.qk_norm_rope(t, t, i, torch.zeros(64))
    with pytest.raises(ValueError, match="CUDA device"):
        fwlib.paged_prefill(t, t, t, i, i, i, 0.1)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        fwlib.verify_drafts([1], [2], [3], [4])
    with pytest.raises(TypeError, match="tokens is required"):
        fwlib.verify_drafts(None, None, None, None)

