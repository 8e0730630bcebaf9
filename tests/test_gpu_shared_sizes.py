"""Attention over groups at the sizes that lie between its paths: every page size, calls of many tokens and few rows, long rows among
many, pools past 32 bits.  Against the definition in 64 bits; tolerances: ``kv_reference.attention_tolerance``."""
import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests import kv_reference as ref
from tests.test_gpu_attention import BF16, F32, i32
from tests.test_gpu_shared import Groups

pytestmark = pytest.mark.gpu

PREFIXES = [(600, [(1, 601), (2, 700), (1, 950)]), (300, [(3, 310), (1, 550)]), (256, [(1, 257), (4, 300)])]


def bits(max_q, group, dim, dtype):
    """Those that are kept: 16 in calls without a row of more than 64 queries per kv-head, 8 in others (24 on the CUDA cores)."""
    return 24 if dtype == F32 or dim == 96 else 16 if max_q * group <= 64 else 8


@pytest.fixture
def keep(monkeypatch):
    def of(n):
        monkeypatch.setattr("tests.test_gpu_shared.weight_bits", lambda dim, dtype: n)
    return of


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (256, BF16), (96, BF16), (64, F32)])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 5)])
def test_pages_of_every_size(keep, page, window, sinks, dim, dtype):
    keep(bits(4, 4, dim, dtype))
    null = [(1, e, 0) for e in (0, 2)] if page < 256 else []
    Groups(PREFIXES, lone=[(1, 270), (2, 40)], heads=8, dim=dim, dtype=dtype, page=page, window=window, sinks=sinks, null=null,
           seed=page).check()


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (256, BF16), (64, F32)])
@pytest.mark.parametrize("window", [0, 60])
def test_more_tokens_than_a_pass_plans_itself(keep, window, dim, dtype):
    """200 rows of 6 tokens."""
    keep(bits(6, 2, dim, dtype))
    groups = [(96, [(6, 104 + i) for i in range(20)]) for _ in range(10)]
    Groups(groups, heads=4, dim=dim, dtype=dtype, window=window, sinks=3, seed=1).check()


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (256, BF16), (64, F32)])
@pytest.mark.parametrize("window", [0, 60])
def test_long_rows_among_many(keep, window, dim, dtype):
    """The plan's kernel places long rows' tokens a warp each."""
    keep(bits(128, 1, dim, dtype))
    groups = [(96, [(70, 170), (1, 104), (128, 230), (3, 120)])] + [(16, [(1, 20), (2, 19)])] * 140
    Groups(groups, heads=2, dim=dim, dtype=dtype, window=window, sinks=3, seed=2).check()


@pytest.mark.parametrize("new,dim,dtype", [(1, 64, BF16), (3, 128, BF16), (60, 128, BF16), (2, 256, BF16), (1, 96, BF16), (3, 64, F32)])
def test_offsets_past_32_bits(new, dim, dtype):
    """Pages whose element offsets pass 2^31: K and V in one allocation of a little over 2^32 elements."""
    heads, page = 4, 256
    per = 2 * heads * page * dim
    pages = (1 << 32) // per + 9
    both = torch.empty(pages, 2, heads, page, dim, dtype=dtype, device="cuda")
    kv = 2 * page + 77
    ids = [[pages - 1, pages // 2 + 1, pages - 3], [pages - 1, pages // 2 + 1, pages - 4]]
    gen = torch.Generator().manual_seed(dim)
    small = torch.zeros(5, 2, heads, page, dim, dtype=dtype)
    small[1:] = torch.randn(4, 2, heads, page, dim, generator=gen).to(dtype)
    for i, p in enumerate(ids[0] + ids[1][2:]):
        both[p] = small[i + 1].cuda()
    q = torch.randn(2 * new, heads, dim, generator=gen).to(dtype)
    rows = gdn.KvRows(i32([0, new, 2 * new]), 2 * new, i32([kv, kv]), new)
    cache = gdn.KvCache(both[:, 0], both[:, 1], i32(ids))
    groups = gdn.KvGroups(i32([0, 2]), i32([0]))
    qd, out, status = q.cuda(), torch.empty(2 * new, heads, dim, dtype=dtype, device="cuda"), i32([0])
    gdn.gdn_kv_common_prefix(cache, rows, groups, status=status)
    shared = min(2 * page, (kv - new) // page * page)
    assert groups.prefix_lens.tolist() == [shared]
    gdn.gdn_shared_attention(gdn.Attention(heads), cache, rows, groups, qd, out, status=status)
    want, spread, logits = ref.attention(q, small[:, 0], small[:, 1], torch.tensor([[1, 2, 3], [1, 2, 4]]), [(0, new), (new, new)],
                                         [0, 1], list(range(2 * new)), [kv, kv], 0.0, 0, 0)
    tol = ref.attention_tolerance(want, spread, logits, kv, dim, dtype, bits(new, 1, dim, dtype))
    assert torch.all((out.cpu().double() - want).abs() <= tol)
    k = torch.randn(2 * new, heads, dim, generator=gen).to(dtype).cuda()
    rope, turned = gdn.Rope(dim), torch.empty_like(k)
    positions = [kv - new + t for t in range(new)] * 2
    gdn.gdn_rope(rope, i32(positions), k, turned)
    gdn.gdn_kv_append_rope(cache, rows, rope, k, -k, status=status)
    assert int(status) == 0
    for t, pos in enumerate(positions):
        p = ids[t // new][pos // page]
        assert torch.equal(both[p, 0, :, pos % page], turned[t]) and torch.equal(both[p, 1, :, pos % page], -k[t])
