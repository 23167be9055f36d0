"""Page tables beside a request whose counts contradict each other by the most 32
bits hold: the others' slots, pages and offsets are those of the definition."""
import pytest

from tests.gpu_common import built_library
from tests.test_spec_tables_gpu import run_tables, table_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,ps,L", [(6, 32, 2), (300, 16, 8), (2284, 1, 12), (3000, 16, 96), (7, 16, 0), (2500, 16, 0)])
@pytest.mark.parametrize("name", ["new_lens", "seq_lens", "held"])
@pytest.mark.parametrize("value", [2 ** 31 - 1, -2 ** 31])
def test_counts_at_the_ends_of_32_bits(name, value, B, ps, L, in_place):
    x = table_case(B, ps, L, seed=B, leave=0.0)
    for b in {0, B // 3, B // 3 + 1, B // 2}:
        x[name][b] = value
    run_tables(built_library(), x, status=1, in_place=in_place)
