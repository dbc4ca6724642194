"""Page calls on a cache of no pages: what is wrong with the table is recorded all the same."""
import pytest

import kda_linear_attention_bounded_gb300 as kda
from test_pages_gpu import compact, release

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,status", [
    ([0, 0], 0), ([-1, 0], kda.KDA_DEVICE_BAD_COUNT), ([0, 33], kda.KDA_DEVICE_BAD_COUNT), ([5, 0], kda.KDA_DEVICE_BAD_PAGE),
    ([5, -2], kda.KDA_DEVICE_BAD_COUNT | kda.KDA_DEVICE_BAD_PAGE)])
def test_findings_of_an_empty_cache(lens, status):
    table = [[0, 3], [-1, 0]]
    assert release(table, lens, [-1], 16, 0) == (lens, [], 0, status)
    got, found = compact(table, lens, 16, 0, 2, in_place=True)
    assert got == (table, [-1, -1], [-1, -1], [], 0) and found == status
