"""Norms of heads at the ends of FP32's range.  Bounds: those of test_norm_rope_gpu."""
import pytest
import torch

from tests import test_norm_rope_gpu as rope
from tests.gpu_common import built_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    return built_library()


def heads(exponents, D, seed=0):
    """A token to an exponent; its elements lie between it and the next."""
    g = torch.Generator().manual_seed(seed)
    sign = torch.randint(0, 2, (len(exponents), 2, D), generator=g) * 2 - 1
    x = sign * (1 + torch.rand(len(exponents), 2, D, generator=g)).double()
    x = torch.where(x.abs() >= 1.99, x.sign() * 1.5, x)          # no element rounds up to the next binade
    x = (x * 2.0 ** torch.tensor(exponents).double()[:, None, None]).to(torch.bfloat16).cuda()
    freq = (1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    pos = torch.arange(len(exponents), dtype=torch.int32, device="cuda") * 7 + 3
    return dict(q=x, k=x.clone(), positions=pos, inv_freq=freq, axis_map=None)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_heads_that_are_normed_to_the_full(fw, D):
    w = torch.full((D,), 1.5, device="cuda")
    x = dict(heads([-60, -40, -1, 0, 30, 57, 58], D), q_weight=w, k_weight=None, eps=0.0)
    q, k = fw.qk_norm_rope(**x)
    rope.check_bf16(q, rope.want(x, "q"), "q")
    rope.check_bf16(k, rope.want(x, "k"), "k")               # not normed: as large as they are
    assert fw.device_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_heads_whose_squares_are_too_many(fw, D):
    """Zeros; NaN where the product with the weight is past FP32."""
    x = dict(heads([61, 64, 100, 124, 3], D), q_weight=torch.ones(D, device="cuda"), k_weight=torch.full((D,), 64.0, device="cuda"),
             eps=1e-6)
    q, k = fw.qk_norm_rope(**x)
    assert (q[:4] == 0).all() and (k[:3] == 0).all() and torch.isnan(k[3]).any()
    ref = rope.want(x, "q")
    rope.check_bf16(q[4:], (ref[0][4:], ref[1][4:]), "q")
