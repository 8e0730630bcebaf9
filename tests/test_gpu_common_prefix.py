"""The common prefix where rows leave one another in many places at once."""
import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests.test_gpu_attention import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,entries,groups", [(5, 40, 3), (16, 300, 2), (60, 1000, 1), (24, 8192, 16), (200, 8192, 1), (64, 4096, 4)])
def test_every_row_leaves_at_a_place_of_its_own(rows, entries, groups):
    """Warps end their search while others, and their own lanes, still lower what they look at."""
    gen = torch.Generator().manual_seed(rows)
    first = torch.randint(1, 1000, (groups, entries), generator=gen, dtype=torch.int32)
    pool = torch.zeros(1001, 1, 16, 16, device="cuda")
    n = rows * groups
    kv_rows = gdn.KvRows(i32(list(range(n + 1))), n, i32([entries * 16] * n), 1)
    of_groups = gdn.KvGroups(i32([g * rows for g in range(groups + 1)]), i32([-7] * groups))
    status = i32([0])
    for i in range(20):
        table = first.repeat_interleave(rows, 0)
        # late places first, so that many are found, and some tables that part near their end alone
        low = 0 if i % 2 else entries * 3 // 4
        at = torch.randint(low, entries - 1, (n,), generator=gen)
        at[::rows] = entries  # (a group's first row is what the others are compared with)
        member = (at < entries).nonzero()[:, 0]
        table[member, at[member]] = 1000
        cache = gdn.KvCache(pool, pool, table.cuda())
        for _ in range(5):
            of_groups.prefix_lens.fill_(-7)
            gdn.gdn_kv_common_prefix(cache, kv_rows, of_groups, status=status)
            assert of_groups.prefix_lens.tolist() == [16 * int(p.min()) for p in at.view(groups, rows)]
    assert int(status) == 0
