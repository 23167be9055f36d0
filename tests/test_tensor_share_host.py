"""The test for common elements of two strided tensors (csrc/tensor_share.h),
compiled for the host, against all addresses written out."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

from tests.test_abi_host import fake

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32, I32, E4M3 = 0, 1, 2, 3
SIZE = {BF: 2, F32: 4, I32: 4, E4M3: 1}


@pytest.fixture(scope="module")
def share(tmp_path_factory):
    d = tmp_path_factory.mktemp("share")
    src = d / "share.cpp"
    src.write_text('#include "tensor_share.h"\n'
                   'extern "C" int share(const fw_tensor_t *a, int64_t ea, const fw_tensor_t *b, int64_t eb) {\n'
                   '    return fw::tensors_share(a, ea, b, eb);\n}\n')
    lib = d / "share.so"
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"),
                           "-I", os.path.join(ROOT, "ragged_softmax_attention_gb300", "csrc"), str(src), "-o", str(lib)])
    f = ctypes.CDLL(str(lib)).share
    f.argtypes = [ctypes.c_void_p, ctypes.c_int64] * 2
    return lambda a, b: bool(f(ctypes.addressof(a), SIZE[a.dtype], ctypes.addressof(b), SIZE[b.dtype]))


def held(t):
    e = SIZE[t.dtype]
    out = set()
    for idx in itertools.product(*(range(t.shape[i]) for i in range(t.ndim))):
        at = t.data + e * sum(i * t.stride[k] for k, i in enumerate(idx))
        out.update(range(at, at + e))
    return out


def test_against_all_addresses(share):
    r = random.Random(1)
    yes = 0
    for _ in range(3000):
        ts = []
        common = sorted(r.choice([0, 1, 2, 3, 5, 8, 12, 24, 40, 64]) for _ in range(3))[::-1]
        for _ in range(2):
            nd = r.randint(1, 4)
            strides = (common if r.random() < 0.5 else [r.randint(0, 40) for _ in range(3)])[:nd - 1] + [1]
            shape = [r.randint(1, 4) for _ in range(nd)]
            if r.random() < 0.05:
                shape[r.randrange(nd)] = 0
            ts.append(fake(shape, r.choice([BF, F32, I32, E4M3]), ptr=0x1000 + 4 * r.randint(0, 60), strides=strides))
        want = bool(held(ts[0]) & held(ts[1]))
        assert share(ts[0], ts[1]) == want == share(ts[1], ts[0])
        yes += want
    assert 500 < yes < 2500


def test_views_of_one_buffer(share):
    """Interleaved extents, nothing in common: columns of a fused projection, page
    halves, and one place further each."""
    row = (40 + 8 + 8) * 128
    q = fake([64, 32, 40, 128], BF, 0x100000, [32 * row, row, 128, 1])
    k = fake([64, 32, 8, 128], BF, 0x100000 + 40 * 128 * 2, [32 * row, row, 128, 1])
    assert not share(q, k)
    k.data -= 2
    assert share(q, k)
    page = 16 * 8 * 128
    kc = fake([30000, 16, 8, 128], BF, 0x100000, [2 * page, 8 * 128, 128, 1])
    vc = fake([30000, 16, 8, 128], BF, 0x100000 + 2 * page, [2 * page, 8 * 128, 128, 1])
    assert not share(kc, vc)
    vc.data += 2 * 29999 * 2 * page
    assert not share(kc, vc)
    vc.data -= 2
    assert share(kc, vc)
    lse = fake([64, 32, 40], F32, 0x100000, [32 * 40, 40, 1])
    assert share(lse, fake([64, 32, 40, 128], BF, 0x100000 - 2))
    # strides that fit nothing: given up, and taken for shared
    assert share(fake([5000, 5000], I32, 0x100000, [7919, 1]), fake([5000, 5000], I32, 0x100000, [10007, 1]))
