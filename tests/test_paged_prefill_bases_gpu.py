"""Chunk attention while the base of the exponentials moves: scores that rise tile after tile,
by other amounts in every row, so that O is read, scaled and written back in the middle of a
piece.  For one row tile a request, where several key tiles are on their way at once, as well
as for two.  Bounds: those of test_paged_prefill_gpu."""
import pytest
import torch

from tests import test_paged_prefill_gpu as chunk
from tests.gpu_common import built_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    return built_library()


def rising(d, n, Hq, Hkv, D, ps, kv8, shape, seed):
    """Element 0 carries the trend: up to 10 a tile of 128 keys in the natural exponent
    (14 in base 2, more than the 8 that the base is let behind), times a factor of the row
    between a quarter and one."""
    x = chunk.make(d, n, Hq, Hkv, D, ps, kv8=kv8, seed=seed)
    g = torch.Generator().manual_seed(seed)
    x["k_scale"] = 0.5 if kv8 else 1.0
    per_tile = 10.0 / (16.0 * x["scale"] * x["k_scale"])
    k = x["k_cache"].float() * (0.02 if kv8 else 0.5)
    for b, length in enumerate(n):
        at = torch.arange(length)
        tile = (at // 128).float()
        level = tile if shape == "rising" else tile.max() - tile if shape == "falling" else \
            torch.rand(length, generator=g) * tile.max()
        pages = x["block_table"][b].long()[at // ps]
        k[pages, at % ps, :, 0] = (level * per_tile)[:, None]
    assert not kv8 or k.nan_to_num().abs().max() < 448
    x["k_cache"] = k.to(x["k_cache"].dtype)
    x["q"][..., 0] = (16.0 * (0.25 + 0.75 * torch.rand(x["q"].shape[:2], generator=g))).to(torch.bfloat16)
    return x


@pytest.mark.parametrize("ctas", [0, 1])                  # pieces of a few tiles, and all of a unit in one
@pytest.mark.parametrize("shape", ["rising", "falling", "scattered"])
@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
@pytest.mark.parametrize("d,n,Hq,Hkv", [([8], [2900], 4, 2), ([1, 30, 3], [2000, 1300, 700], 4, 1), ([150], [2000], 4, 2)])
def test_bases_that_move(fw, d, n, Hq, Hkv, D, kv8, shape, ctas):
    fw.set_option(fw.FW_OPT_MAX_CTAS, ctas)
    try:
        chunk.run_and_check(fw, rising(d, n, Hq, Hkv, D, 16, kv8, shape, 40 + len(d)), f"{d} {shape}")
    finally:
        fw.set_option(fw.FW_OPT_MAX_CTAS, 0)
