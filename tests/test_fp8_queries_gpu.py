"""Queries over 8-bit caches, whose rows are carried as two E4M3 terms on a power of two of
their own: exact for every element down to 2^-9 of the row's largest, within 2^-17 of it
below.

A single key that is one in one place makes a row's LSE the element there, times the
scale: score, exponent and natural logarithm cost FP32 roundings, under 2^-21 of it.  The
decodes take their weights as FP16 with a power of two in front (2^7, or their headroom), which
the LSE takes back: in base 2 the exponential of 7 is off by 2^-22 of itself (2^-21.5 of a
logarithm), a logarithm of 7 by 2 ulp (2^-20), and two sums of up to 8 by half an ulp each (2^-21
together): under 2^-19.3, times ln 2, under 2^-19.  (What two terms lose below 2^-9, 2^-17
of the largest times the scale, is up to 2^-17.5.)"""
import math

import pytest
import torch

from tests.gpu_common import built_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    return built_library()


def rows():
    """(largest, element): every mantissa of three binades below three largest magnitudes,
    which lie at the beginning, in the middle and at the end of theirs."""
    m = 1 + torch.arange(128, dtype=torch.float64) / 128
    out = [torch.stack([torch.full_like(m, top), sign * m * 2.0 ** e], -1)
           for top in (1.0, 1.5, 1.9921875) for e in (-8, -9, -10) for sign in (1, -1)]
    return torch.cat(out)


@pytest.mark.parametrize("entry", ["paged_prefill", "one row tile", "paged_decode_tree", "paged_decode_fp8"])
def test_two_terms_hold_an_element(fw, entry):
    x = rows()
    N, D, ps, scale = x.shape[0], 128, 16, 0.7
    assert (x.to(torch.bfloat16).double() == x).all()
    q = torch.zeros(N, 1, D, dtype=torch.bfloat16)
    q[:, 0, 40], q[:, 0, 5] = x[:, 0].to(torch.bfloat16), x[:, 1].to(torch.bfloat16)
    k = torch.zeros(1, ps, 1, D)
    k[0, 0, 0, 5] = 1.0
    k, v = k.to(torch.float8_e4m3fn).cuda(), torch.ones(1, ps, 1, D).to(torch.float8_e4m3fn).cuda()
    q = q.cuda()
    i32 = lambda t: torch.as_tensor(t, dtype=torch.int32).cuda()
    if entry == "paged_prefill":
        lse = fw.paged_prefill(q, k, v, i32([[0]]), i32([0, N]), i32([1]), scale, causal=False)[1]
    elif entry == "one row tile":                         # a request to a token
        lse = fw.paged_prefill(q, k, v, i32(torch.zeros(N, 1)), i32(torch.arange(N + 1)), i32(torch.ones(N)), scale)[1]
    elif entry == "paged_decode_tree":
        mask = fw.tree_mask(i32(torch.full((N, 1), -1)))[0]
        lse = fw.paged_decode_tree(q[:, None], k, v, i32(torch.zeros(N, 1)), i32(torch.ones(N)), mask, scale)[1]
    else:
        lse = fw.paged_decode_fp8(q[:, None], k, v, i32(torch.zeros(N, 1)), i32(torch.ones(N)), scale, 1.0, 1.0)[1]
    assert fw.device_status() == 0
    got, want = lse.double().cpu().reshape(N), scale * x[:, 1]
    exact = x[:, 1].abs() >= 2.0 ** -9 * x[:, 0]
    assert 256 < int(exact.sum()) < N
    err = (got - want).abs()
    room = 2.0 ** -21 * want.abs() + (2.0 ** -19 if "decode" in entry else 0.0)
    assert (err <= room)[exact].all()
    assert (err <= room + scale * 2.0 ** -17 * x[:, 0])[~exact].all()
    assert math.isfinite(float(err.max()))
