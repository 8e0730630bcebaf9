"""Page calls at the limits of a descriptor."""
import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [64, 131073])
def test_needs_whose_sum_passes_32_bits(pages):
    """2100 rows that lack 2^20 entries each, as many as a row may have, between two rows of few: the sum of needs
    passes 2^31, and no row behind the first gets a page."""
    rows, width = 2102, 1 << 20
    pool = torch.zeros(pages, 1, 16, 16, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(rows, width, dtype=torch.int32, device="cuda")  # 8.8 GB
    count = torch.zeros(pages, dtype=torch.int32, device="cuda")
    cache = gdn.KvCache(pool, pool, table, count)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    zeros = torch.zeros(rows, dtype=torch.int32, device="cuda")
    to = torch.full_like(zeros, 16 * width)
    to[0], to[-1] = 40, 16
    gdn.gdn_kv_reserve(cache, None, zeros, to, status=status)
    assert int(status) == ref.NO_PAGES
    assert table[0, :4].tolist() == [1, 2, 3, 0]
    assert int(table[0].count_nonzero()) == 3
    assert all(int(table[i:i + 256].count_nonzero()) == 0 for i in range(1, rows, 256))
    assert count[:5].tolist() == [0, 1, 1, 1, 0] and int(count.sum()) == 3
