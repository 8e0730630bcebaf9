"""Prompts whose scores grow along the cache, so that the maximum that the weights refer to moves, with values of
ordinary and of very large size.  Tolerances: ``kv_reference.attention_tolerance``."""
import pytest
import torch

from tests.test_gpu_attention import Step

pytestmark = pytest.mark.gpu

CUT = dict(rows=[(300, 700), (90, 333)], heads=8, kv_heads=2)                        # items cut into pieces
WHOLE = dict(rows=[(700, 700), (1, 9), (641, 1100), (130, 130)], heads=16, kv_heads=16)  # a CTA takes whole ones


def growing(slope, size, dim, rows, seed, **kw):
    """A step whose score of position j is about slope * j (in nats), and whose values are of about ``size``."""
    s = Step(rows, dim=dim, page=32, seed=seed, **kw)
    gen = torch.Generator().manual_seed(seed + 1)
    u = torch.randn(s.kv_heads, dim, generator=gen)
    u /= u.norm(dim=-1, keepdim=True)
    k, v = s.k.float(), s.v.float()
    for i, (_, kv) in enumerate(s.rows):
        j = torch.arange(kv)
        page, slot = s.table[s.table_rows[i]].long()[j // s.page], j % s.page
        k[page, :, slot] = 0.25 * k[page, :, slot] + slope * j[:, None, None] * u
        v[page, :, slot] = size * v[page, :, slot]
    q = 0.1 * s.q.float() + dim ** 0.5 * u.repeat_interleave(s.heads // s.kv_heads, 0)
    s.k, s.v, s.q = k.to(s.dtype), v.to(s.dtype), q.to(s.dtype)
    s.kv[0].copy_(s.k)
    s.kv[1].copy_(s.v)
    s.qd.copy_(s.q)
    return s


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("items", [CUT, WHOLE], ids=["cut", "whole"])
@pytest.mark.parametrize("slope", [0.05, 0.35, -0.1])  # 5, 32, -9 powers of two per 64 tokens
def test_scores_that_grow_along_the_cache(slope, items, dim):
    growing(slope, 1.0, dim, seed=dim, **items).check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("items", [CUT, WHOLE], ids=["cut", "whole"])
@pytest.mark.parametrize("slope", [0.05, 0.35])
def test_large_values_under_growing_scores_stay_finite(slope, items, dim):
    growing(slope, 2.0 ** 100, dim, seed=dim + 1, **items).check()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scores_that_grow_in_a_window(dim):
    growing(0.35, 2.0 ** 90, dim, [(300, 700), (200, 1500)], heads=4, kv_heads=2, seed=dim + 2, window=200, sinks=9).check()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_the_same_rows_one_token_at_a_time(dim):
    """Decode rows over the same caches: the other kernel, the same formula."""
    growing(0.05, 2.0 ** 100, dim, [(1, 700), (2, 333)], heads=8, kv_heads=2, seed=dim + 1).check()
