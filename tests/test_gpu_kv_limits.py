"""Page calls at the limits of a descriptor."""
import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests import kv_reference as ref
from tests.test_gpu_attention import BF16, F32, Step
from tests.test_gpu_kv_pages import Pool

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


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (256, BF16), (96, BF16), (64, F32)])
def test_rows_longer_than_a_length_of_zero_are_reported(dim, dtype):
    s = Step([(1, 20), (0, 7), (3, 40)], dim=dim, dtype=dtype, gather=False)
    s.kv_rows = gdn.KvRows(s.kv_rows.query_start_loc, 4, s.kv_rows.kv_lens, 0, s.kv_rows.table_rows)
    got, status = s.run()
    assert status == ref.ROW_RANGE and torch.all(got.float() == 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.ones(4, 2, dim, dtype=dtype, device="cuda")
    before = [t.clone() for t in s.kv]
    gdn.gdn_kv_append(s.cache, s.kv_rows, k, k, status=status)
    assert int(status) == ref.ROW_RANGE
    view = torch.int16 if dtype == BF16 else torch.int32
    assert all(torch.equal(a.view(view), b.view(view)) for a, b in zip(s.kv, before))


@pytest.mark.parametrize("width", [1023, 1024, 1025, 2500])
@pytest.mark.parametrize("pages", [9000, 131073])
def test_forks_in_tables_of_long_rows(width, pages):
    """Tables of up to 1024 entries a row and of more: other launches, the same pages."""
    P = Pool(pages, 12, width, page=16, heads=2, dim=16)
    full = 16 * width
    P.reserve([3, 8, 0], [0, 0, 0], [full, full - 5, 100])
    P.fork([3, 8, 3, 8, 0, 3], [1, 2, 4, 5, 6, 7], [full, full - 5, 33, full - 16, 100, full - 1])
    P.same()
    assert P.ref.status == 0
    P.fork([1, 2], [9, 10], [full - 7, 500])
    P.same()
    P.release([3, 8, 1], [0, 5, 0], [width, width, 7])
    P.fork([2, 9, 5], [3, 8, 11], [full - 5, full - 7, 0])
    P.same()
    assert P.ref.status == ref.PAGE_RANGE  # row 8 still holds its first pages
