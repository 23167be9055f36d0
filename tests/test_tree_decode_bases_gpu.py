"""Tree decode where the base of a row's exponentials moves, where the score
factor vanishes, and where one key carries a row, over every kind of cache and
on both sides of 128 rows.

Bounds, beside those of test_tree_decode_gpu.py: over an 8-bit cache a weight is
rounded to FP16, half a step 2^-11 of it, against a row sum of unrounded ones.
It carries 2^7 over a base that the row's largest weight is never below, so
weights under 2^-14 / 2^7 of that are off by half a subnormal step, 2^-25, each:
n keys move an output by at most n * 2^-32 * max |v|.
"""
import math

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


def capped(fw, ctas, call):
    fw.set_option(fw.FW_OPT_MAX_CTAS, ctas)
    try:
        return call()
    finally:
        fw.set_option(fw.FW_OPT_MAX_CTAS, 0)


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


@pytest.mark.parametrize("ctas", [0, 1])       # rows cut into pieces, and kept whole
@pytest.mark.parametrize("scale", [-0.7, 0.0, 1.5])
@pytest.mark.parametrize("T,Hq,Hkv", ROWS)
@pytest.mark.parametrize("D,kv8", KINDS)
def test_scales(fw, D, kv8, T, Hq, Hkv, scale, ctas):
    x = make(2, T, Hq, Hkv, D, 32, [1100, 390], [T, T - 3], "tree", kv8=kv8, seed=71)
    x["scale"] = scale
    capped(fw, ctas, lambda: run_tight(fw, x, f"scale {scale}"))


@pytest.mark.parametrize("ctas", [0, 1])
@pytest.mark.parametrize("turn", [1, -1])
@pytest.mark.parametrize("T,Hq,Hkv", ROWS)
@pytest.mark.parametrize("D,kv8", KINDS)
def test_scores_that_rise_in_every_tile(fw, D, kv8, T, Hq, Hkv, turn, ctas):
    """All queries near one direction, keys along it that grow by some 9 log2 units a
    tile (turn 1), or against it under a negative scale (turn -1)."""
    n, ps = 1500, 64
    x = make(1, T, Hq, Hkv, D, ps, [n], None, "tree", kv8=kv8, seed=73)
    g = torch.Generator().manual_seed(74)
    u = torch.randn(D, generator=g)
    u *= math.sqrt(D) / u.norm()
    x["q"] = (u + 0.2 * torch.randn(1, T, Hq, D, generator=g)).to(torch.bfloat16)
    grow = torch.linspace(0, 70.0 / math.sqrt(D), n)           # score = grow * D / sqrt(D)
    pages = x["block_table"][0, :-(-n // ps)].long()
    k = torch.zeros(len(pages) * ps, Hkv, D)
    k[:n] = (turn * grow[:, None, None] * u + 0.05 * torch.randn(n, Hkv, D, generator=g)) / x["k_scale"]
    if kv8:
        k.clamp_(-448, 448)
    x["k_cache"][pages] = k.view(len(pages), ps, Hkv, D).to(x["k_cache"].dtype)
    x["scale"] *= turn
    capped(fw, ctas, lambda: run_tight(fw, x, "rising scores"))


@pytest.mark.parametrize("ctas", [0, 1, 3])
@pytest.mark.parametrize("T,Hq,Hkv", [(30, 8, 2), (60, 8, 2)])
@pytest.mark.parametrize("D,kv8", KINDS)
def test_one_key_carries_a_row(fw, D, kv8, T, Hq, Hkv, ctas):
    """Every row's weight lies on a key of its own, next to an edge of a page, of half a
    tile, of a tile or of a piece: a value taken from elsewhere, or cleared, shows."""
    n, ps = 64 * T + 21, 32
    x = make(1, T, Hq, Hkv, D, ps, [n], None, "tree", kv8=kv8, seed=77)
    base, G = n - T, Hq // Hkv
    k = x["k_cache"]
    for t in range(T):
        for h in range(Hq):
            # the keys before and behind place 64 t and 64 t + 32, a row each
            j = min(max(0, 64 * t + (h % G >> 1) * 32 - (h & 1)), base - 1)
            page, off = int(x["block_table"][0, j // ps]), j % ps
            key = x["q"][0, t, h].float() * 4.0 / x["k_scale"]
            k[page, off, h // G] = (key.clamp(-448, 448) if kv8 else key).to(k.dtype)
    ref = spec.tree_attention(**x)
    assert (np.abs(ref[0]).max(-1) > 0.5 * ref[2].max(-1)).mean() > 0.9      # one key's value, not an average
    capped(fw, ctas, lambda: run_tight(fw, x, "one key"))


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


@pytest.mark.parametrize("turn", [1, -1])
@pytest.mark.parametrize("T,Hq,Hkv", ROWS)
@pytest.mark.parametrize("D,kv8", KINDS)
def test_small_scales_of_large_scores(fw, D, kv8, T, Hq, Hkv, turn):
    """Queries and keys of large magnitudes under a scale that undoes them."""
    x = make(2, T, Hq, Hkv, D, 32, [700, T], None, "tree", kv8=kv8, seed=83)
    x["q"] *= 2.0 ** (110 if kv8 else 58)
    if not kv8:
        x["k_cache"] *= 2.0 ** 52
    x["scale"] *= turn * 2.0 ** -110
    run_tight(fw, x, "large scores")


@pytest.mark.parametrize("T,Hq,Hkv", ROWS)
@pytest.mark.parametrize("D,kv8", KINDS)
def test_orders_of_dimensions(fw, D, kv8, T, Hq, Hkv):
    """Caches with a page's heads before its slots, queries with heads before drafts,
    outputs and LSE with the batch last."""
    x = make(3, T, Hq, Hkv, D, 32, [700, T, 130], [T, T, T - 2], "tree", kv8=kv8, seed=85)
    g = on_gpu(x)
    for name in ("k_cache", "v_cache"):
        raw = g[name].view(torch.uint8) if kv8 else g[name]
        g[name] = raw.permute(0, 2, 1, 3).contiguous().view(g[name].dtype).permute(0, 2, 1, 3)
    g["q"] = g["q"].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    plain = fw.paged_decode_tree(**on_gpu(x))
    out = torch.full((Hq, T, 3, D), 7.0, dtype=torch.bfloat16, device="cuda").permute(2, 1, 0, 3)
    lse = torch.full((T, 3, Hq), 7.0, device="cuda").permute(1, 0, 2)
    fw.paged_decode_tree(**g, out=out, lse=lse)
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])


@pytest.mark.parametrize("T,Hq,Hkv", ROWS)
@pytest.mark.parametrize("D,kv8", KINDS)
def test_scale_zero_of_the_largest_queries(fw, D, kv8, T, Hq, Hkv):
    """Every visible key weighs the same whatever the magnitude of the queries."""
    x = make(3, T, Hq, Hkv, D, 32, [700, T, 130], [T, T, T - 2], "tree", kv8=kv8, seed=87)
    x["q"] *= 2.0 ** (125 if kv8 else 115)                 # BF16 scores stay finite in FP32
    x["scale"] = 0.0
    assert torch.isfinite(x["q"]).all()
    run_tight(fw, x, "largest queries")
