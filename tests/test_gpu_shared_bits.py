"""Attention over groups keeps as many bits of the weights as attention without groups: 16 of every row of up to 64 queries per
kv-head, whatever the groups share.  Against the definition in 64 bits; tolerances: ``kv_reference.attention_tolerance``."""
import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests import test_gpu_shared as shared
from tests.test_gpu_attention import i32
from tests.test_gpu_shared import TREE, Groups

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def sixteen_bits(monkeypatch):
    monkeypatch.setattr(shared, "weight_bits", lambda dim, dtype: 16)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
def test_groups(dim, page, window, sinks):
    Groups(TREE, lone=[(1, 50), (2, 2)], dim=dim, page=page, seed=dim, heads=8, window=window, sinks=sinks).check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,new", [(8, 1), (64, 1), (16, 4), (4, 32)])
def test_up_to_64_queries_of_a_row(dim, heads, new):
    groups = [(700, [(new, 800), (1, 750), (new, 900)]), (100, [(new, 100 + new)] * 5)]
    Groups(groups, dim=dim, heads=heads, kv_heads=1 if heads == 64 else 2, seed=heads).check()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_nothing_is_shared(dim):
    s = Groups([(200, [(1, 230), (3, 260), (1, 300)])], dim=dim, heads=8, seed=3)
    s.groups = gdn.KvGroups(s.groups.group_start_loc, i32([0]))
    s.check()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_decode_rows_beside_a_longer_one(dim):
    """A call that attention without groups takes both ways: its short rows keep 16 bits there."""
    groups = [(128, [(1, 140 + i) for i in range(9)] + [(33, 200)])]
    Groups(groups, dim=dim, heads=4, kv_heads=2, seed=4).check()


@pytest.mark.parametrize("heads,dim", [(4, 64), (4, 128), (4, 256), (64, 128)])
def test_values_that_are_not_finite(heads, dim):
    """Tokens that hold infinities go by another way, with the same weights."""
    shared.test_values_that_windows_hide(heads, dim, torch.bfloat16)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_that_cancel(dim):
    """Keys in pairs that differ by little, values in pairs of opposite sign: a weight's lost bits would stay."""
    s = Groups([(512, [(1, 530), (2, 600)])], dim=dim, heads=8, gather=False, seed=8)
    for page in range(1, s.k.shape[0]):
        s.k[page, :, 1::2] = (s.k[page, :, 0::2].float() * 1.02).to(s.k.dtype)
        s.v[page, :, 1::2] = -s.v[page, :, 0::2]
    s.cache = gdn.KvCache(s.k.cuda(), s.v.cuda(), s.table.cuda())
    s.check()
