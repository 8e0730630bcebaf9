"""Rows whose bounds are none, among good ones: the good ones' results are those of calls without them, whatever makes the plan and
wherever the bad bounds stand.  Against the definition in 64 bits, and the attention without groups."""
import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests import kv_reference as ref
from tests.test_gpu_attention import BF16, F32, i32
from tests.test_gpu_shared import Groups, weight_bits

pytestmark = pytest.mark.gpu


def spoiled(s, starts):
    """Gives the step's rows the bounds ``starts``; returns the rows that are left."""
    total = s.kv_rows.num_tokens
    r = s.kv_rows
    s.kv_rows = gdn.KvRows(i32(starts), total, r.kv_lens, s.max_q, r.table_rows)
    s.starts = starts
    s.rows = [(b - a if 0 <= a <= b <= total and b - a <= min(s.max_q, kv) else 0, kv)
              for a, b, (_, kv) in zip(starts, starts[1:], s.rows)]
    return [i for i, (new, _) in enumerate(s.rows) if new > 0]


def check(s, status=gdn.STATUS_ROW_RANGE):
    want, spread, logits = s.expected()
    tol = ref.attention_tolerance(want, spread, logits, max(kv for _, kv in s.rows), s.dim, s.dtype, weight_bits(s.dim, s.dtype))
    written = torch.zeros(want.shape[0], dtype=torch.bool)
    for i, (new, _) in enumerate(s.rows):
        written[s.starts[i]:s.starts[i] + new] = True
    for attend in (s.run, super(Groups, s).run):  # over groups, and without them
        s.out.fill_(7.0)
        got, said = attend()
        assert said == status
        assert torch.all(got[~written].float() == 7.0)
        bad = ~((got.double() - want).abs() <= tol) & written[:, None, None]
        assert not bad.any(), bad.any(2).any(1).nonzero().flatten().tolist()


TYPES = [(64, BF16), (256, BF16), (96, BF16), (64, F32)]


@pytest.mark.parametrize("dim,dtype", TYPES)
@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("value", [1000000, -5, 0, 1 << 31])
@pytest.mark.parametrize("at", [0, 2, 8, -1])
def test_a_bound_that_is_none(at, value, window, many, dim, dtype):
    groups = [(48, [(1 + i % 2, 50 + i % 7) for i in range(5)]) for _ in range(53 if many else 4)]
    s = Groups(groups, lone=[(1, 20)], heads=2, kv_heads=1, dim=dim, dtype=dtype, window=window, gather=False, seed=at)
    starts = list(s.starts)
    starts[at] = value - (1 << 32) if value >> 31 == 1 else value
    if starts[at] == s.starts[at]:
        return
    left = spoiled(s, starts)
    assert len(left) >= len(s.rows) - 2
    check(s)


@pytest.mark.parametrize("dim,dtype", TYPES)
@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
def test_groups_whose_tokens_lie_between_one_anothers(many, dim, dtype):
    """Group 0's tokens are 4 and 0, group 1's 1 to 3: a row between its rows begins where it should not."""
    s = Groups([(160, [(1, 170), (0, 170), (1, 180)]), (64, [(1, 70), (1, 75), (1, 80)]), (16, [(0, 17)] * (300 if many else 1))],
               heads=2, kv_heads=1, dim=dim, dtype=dtype, gather=False)
    n = len(s.rows)
    s.q = torch.randn(5, 2, dim, generator=torch.Generator().manual_seed(1)).to(dtype)
    s.qd, s.out = s.q.cuda(), torch.full_like(s.q, 7.0, device="cuda")
    s.token = list(range(5))
    r = s.kv_rows
    s.kv_rows = gdn.KvRows(r.query_start_loc, 5, r.kv_lens, 1, r.table_rows)
    s.max_q = 1
    left = spoiled(s, [4, 5, 0, 1, 2, 3] + [4] * (n - 5))
    assert left == [0, 2, 3, 4, 5]
    check(s)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
def test_a_bad_bound_beside_long_rows(many, dtype):
    groups = [(64, [(70, 140), (1, 80), (3, 90), (66, 200)]), (32, [(1, 40), (2, 50)])] + [(16, [(1, 20)] * 2)] * (140 if many else 1)
    s = Groups(groups, heads=2, kv_heads=2, dtype=dtype, gather=False, seed=2)
    starts = list(s.starts)
    starts[2] = -1
    spoiled(s, starts)
    check(s)
