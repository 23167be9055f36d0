"""Tree decode where the score factor vanishes, over every kind of cache and on
both sides of 128 rows.

Bounds, beside those of test_tree_decode_gpu.py: over an 8-bit cache a weight is
rounded to FP16, half a step 2^-11 of it, against a row sum of unrounded ones.
It carries 2^7 over a base that the row's largest weight is never below, so
weights under 2^-14 / 2^7 of that are off by half a subnormal step, 2^-25, each:
n keys move an output by at most n * 2^-32 * max |v|.
"""
import numpy as np
import pytest
import torch

from oracle import spec
from tests.gpu_common import built_library
from tests.test_tree_decode_gpu import U, check, make, on_gpu

pytestmark = pytest.mark.gpu

KINDS = [(128, False), (128, True), (256, False)]
ROWS = [(12, 8, 2), (40, 16, 4)]               # 48 rows of a KV head, and 160


@pytest.fixture(scope="module")
def fw():
    return built_library()


def run_tight(fw, x, what):
    """As run_and_check, with the bound above for the outputs over 8-bit caches."""
    out, lse = fw.paged_decode_tree(**on_gpu(x))
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    ref = spec.tree_attention(**x)
    D = x["q"].shape[-1]
    if x["k_cache"].dtype != torch.float8_e4m3fn:
        check(out, lse, ref, D, what)
        return
    o_ref, _, absv, reach, spread = ref
    check(torch.from_numpy(o_ref), lse, ref, D, what)                        # the LSE
    o = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(o).all(), f"{what}: non-finite output"
    v = x["v_cache"].float()
    vmax = float(v[torch.isfinite(v)].abs().max()) * x["v_scale"]
    delta = (D + 8) * 2.0 ** -24 * reach + 2.0 ** -17 * spread
    d = (2.0 ** -11 + 2 * delta[..., None] + 2.0 ** -18) * absv + int(x["seq_lens"].max()) * 2.0 ** -32 * vmax
    bound = d + U * (np.abs(o_ref) + d) + 1e-30
    diff = np.abs(o - o_ref)
    worst = np.unravel_index(np.argmax(diff / bound), diff.shape)
    assert diff[worst] <= bound[worst], (what, worst, diff[worst], bound[worst], o_ref[worst])


@pytest.mark.parametrize("T,Hq,Hkv", ROWS)
@pytest.mark.parametrize("D,kv8", KINDS)
@pytest.mark.parametrize("what", ["scale", "rows", "tiny", "both", "k_scale"])
def test_score_factors_that_vanish(fw, D, kv8, T, Hq, Hkv, what):
    """Scale zero, queries of zeros and of the least magnitudes, and a vanishing key
    scale: every visible key weighs the same, in tiles that hide keys too."""
    x = make(3, T, Hq, Hkv, D, 32, [700, T, 130], [T, T, T - 2], "tree", kv8=kv8, seed=79)
    if what in ("scale", "both"):
        x["scale"] = 0.0
    if what in ("rows", "both", "k_scale"):
        x["q"][:, ::2] = 0
    if what in ("tiny", "both"):
        x["q"][:, 1::2] *= 2.0 ** -130
    if what == "k_scale":
        x["k_scale"] = 1e-20 if kv8 else 1.0
    run_tight(fw, x, what)
