"""Values that are not finite under chunks at head dim 256, whose row tiles run on a pair of
CTAs: each CTA holds half of the values' columns, and a value that one of them finds makes
the rows of both NaN, run after run."""
import math

import pytest
import torch

from tests import test_paged_prefill_gpu as chunk
from tests.gpu_common import built_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    return built_library()


@pytest.mark.parametrize("column", [0, 100, 127, 128, 255])
@pytest.mark.parametrize("d,n", [([256], [300]), ([256] * 3, [256, 700, 900]), ([256, 140], [261, 150])])
def test_marks_reach_the_rows_of_both_ctas(fw, d, n, column):
    """Heads 1 and 3 hold a bad value in the chunk's first, last but one and middle key in
    turn: every row of theirs that sees it is NaN in all columns, in both row tiles."""
    Hq = 4
    x = chunk.on_gpu(chunk.make(d, n, Hq, Hq, 256, 16, seed=31))
    clean, clean_lse = fw.paged_prefill(**x)
    assert torch.isfinite(clean).all()
    clean_v = x["v_cache"].clone()
    cu = x["cu_seqlens_q"].tolist()
    for back in (255, 2, 128):                            # tokens from the end of a request's chunk
        x["v_cache"].copy_(clean_v)
        want = torch.zeros_like(clean, dtype=torch.bool)
        for b in range(len(d)):
            key = n[b] - min(back, d[b])
            x["v_cache"][x["block_table"][b, key // 16].long(), key % 16, 1::2, column] = math.nan
            want[cu[b] + key - (n[b] - d[b]):cu[b + 1], 1::2] = True
        for _ in range(40):
            out, lse = fw.paged_prefill(**x)
            assert torch.equal(torch.isnan(out), want), f"{back} from the end"
            assert torch.equal(out[~want], clean[~want]) and torch.equal(lse, clean_lse)
    assert fw.device_status() == 0
