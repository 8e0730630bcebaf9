"""Rows whose bounds are none, among good ones: the good ones' results are those of calls without them, whatever makes the plan and
wherever the bad bounds stand.  Against the definition in 64 bits, and the attention without groups."""
import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests import kv_reference as ref
from tests.test_gpu_attention import BF16, F32, i32
from tests.test_gpu_rope import Batch
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


# ------------------------------------------------------------------------------------------
# appending

@pytest.mark.parametrize("turned", [False, True], ids=["append", "append_rope"])
@pytest.mark.parametrize("rows", [9, 100, 3000])
@pytest.mark.parametrize("value", [1000000, -5, 0, 1 << 31])
@pytest.mark.parametrize("at", [0, 2, 5, -2, -1])
def test_append_behind_a_bound_that_is_none(at, value, rows, turned):
    b = Batch([(1 + i % 3, 20 + i % 5) for i in range(rows)], gather=False, seed=rows)
    starts, total = list(b.starts), b.starts[-1]
    starts[at] = value - (1 << 32) if value >> 31 == 1 else value
    if starts == b.starts:
        return
    r = b.kv_rows
    kv_rows = gdn.KvRows(i32(starts), total, r.kv_lens, 3, r.table_rows)
    k, v = torch.full_like(b.k_pool, 5.0), torch.full_like(b.v_pool, 5.0)
    left, places = 0, []
    for i, (lo, hi, (_, kv)) in enumerate(zip(starts, starts[1:], b.rows)):
        if not 0 <= lo <= hi <= total or hi - lo > 3:
            continue
        left += 1
        for t in range(lo, hi):
            pos = kv - (hi - lo) + t - lo
            places.append((t, pos, int(b.table[b.table_rows[i], pos // b.page]), pos % b.page))
    assert left >= rows - 2
    token, pos, page, slot = (list(x) for x in zip(*places))
    status, out = i32([0]), torch.full_like(b.q.contiguous(), 7.0)
    if turned:
        rope = gdn.Rope(64)
        positions = torch.zeros(b.q.shape[0], dtype=torch.int32)
        positions[token] = torch.tensor(pos, dtype=torch.int32)
        want_q, want_k = torch.empty_like(out), torch.empty_like(b.k.contiguous())
        gdn.gdn_rope(rope, positions.cuda(), b.q, want_q)
        gdn.gdn_rope(rope, positions.cuda(), b.k, want_k)
        gdn.gdn_kv_append_rope(b.cache, kv_rows, rope, b.k, b.v, b.q, out, status=status)
        mine = torch.zeros(out.shape[0], dtype=torch.bool, device="cuda")
        mine[token] = True
        assert torch.equal(out[mine], want_q[mine]) and torch.all(out[~mine] == 7.0)
    else:
        want_k = b.k
        gdn.gdn_kv_append(b.cache, kv_rows, b.k, b.v, status=status)
    k[page, :, slot], v[page, :, slot] = want_k[token], b.v[token]
    assert torch.equal(b.k_pool, k) and torch.equal(b.v_pool, v)
    assert int(status) == gdn.STATUS_ROW_RANGE


@pytest.mark.parametrize("turned", [False, True], ids=["append", "append_rope"])
def test_append_of_a_padded_batch(turned):
    """Tokens behind the last row, and rows without tokens at the end, are nobody's."""
    b = Batch([(2, 40), (1, 33), (3, 50), (0, 20), (0, 30)], gather=False)
    r, n = b.kv_rows, b.q.shape[0]
    kv_rows = gdn.KvRows(r.query_start_loc, n, r.kv_lens, 3, r.table_rows)
    status, out = i32([0]), torch.full_like(b.q.contiguous(), 7.0)
    if turned:
        gdn.gdn_kv_append_rope(b.cache, kv_rows, gdn.Rope(64), b.k, b.v, b.q, out, status=status)
        assert torch.all(out[6:] == 7.0) and not torch.any(out[:6] == 7.0)
    else:
        gdn.gdn_kv_append(b.cache, kv_rows, b.k, b.v, status=status)
    written = {(page, slot) for _, _, page, slot in b.positions()}
    for page in range(b.v_pool.shape[0]):
        for slot in range(b.page):
            assert bool(torch.all(b.v_pool[page, :, slot] == 5.0)) == ((page, slot) not in written)
    assert int(status) == 0
