"""Attention calls with more work than the GPU takes at once: several work items for a CTA of the prompt kernel, a last
round that is cut into pieces behind whole ones, more rows than a warp or a CTA looks at in one go.  The 64-bit
reference is computed on the GPU, row by row and head by head.  Tolerances: ``kv_reference.attention_tolerance``."""
import math
import random

import pytest
import torch

from tests import kv_reference as ref
from tests.test_gpu_attention import BF16, F32, Step

pytestmark = pytest.mark.gpu

SMS = 152


def expected(s):
    """``Step.expected`` in products of whole matrices."""
    T, Hq, d = s.q.shape
    G = Hq // s.kv_heads
    scale = s.scale if s.scale > 0 else 1.0 / math.sqrt(d)
    out, spread = (torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda") for _ in range(2))
    logits = torch.zeros(T, Hq, 1, dtype=torch.float64, device="cuda")
    table, q, token = s.table.cuda().long(), s.q.cuda(), torch.tensor(s.token, device="cuda")
    k_pool, v_pool = s.k.cuda(), s.v.cuda()
    for n, (new, kv) in enumerate(s.rows):
        if new == 0:
            continue
        at = token[s.starts[n]:s.starts[n] + new]
        j = torch.arange(kv, device="cuda")
        page, slot = table[s.table_rows[n]][j // s.page], j % s.page
        pos = torch.arange(kv - new, kv, device="cuda")[:, None]
        seen = (j[None] <= pos) & (page > 0)[None]
        if s.window > 0:
            seen &= (j[None] > pos - s.window) | (j[None] < s.sinks)
        for h in range(s.kv_heads):
            k, v = (torch.where((page > 0)[:, None], x[page, h, slot].double(), 0.0) for x in (k_pool, v_pool))
            for g in range(h * G, (h + 1) * G):
                x = q[at, g].double()
                p = torch.softmax((x @ k.T * scale).masked_fill(~seen, -math.inf), -1).nan_to_num(0.0)
                out[at, g], spread[at, g] = p @ v, p @ v.abs()
                logits[at, g] = (x.abs() @ k.abs().T * scale).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
    return out.cpu(), spread.cpu(), logits.cpu()


def check(s, monkeypatch):
    monkeypatch.setattr(s, "expected", lambda: expected(s), raising=False)
    s.check()


def plan(rows, heads, kv_heads, dim, few=0):
    """(whole rounds, items of the last one, pieces of each of those) of the prompt kernel."""
    tile, G = (256 if dim <= 128 else 128), heads // kv_heads
    items = sum(-(-new * G // tile) for new, _ in rows if new * G > few) * kv_heads
    left = items % SMS
    return items // SMS, left, min(16, SMS // left) if left else 1


def test_the_reference_is_the_other_one():
    s = Step([(3, 70), (40, 40), (0, 9)], heads=6, kv_heads=2, dim=64, window=20, sinks=3, null=[(0, 0, 0)], seed=1)
    for a, b in zip(expected(s), s.expected()):
        assert torch.allclose(a, b, rtol=1e-10, atol=1e-12)


LONG = [(2000, 2000), (1300, 1500), (700, 700), (600, 1200), (1, 5)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 333])
@pytest.mark.parametrize("cut", [True, False], ids=["cut", "whole"])
def test_several_rounds_of_items(dim, window, cut, monkeypatch):
    rows = LONG if cut else LONG + [(1024, 1100)]
    rounds, left, pieces = plan(rows, 16, 16, dim)
    assert rounds >= 2 and left > 0 and (pieces > 1) == cut
    check(Step(rows, heads=16, kv_heads=16, dim=dim, page=64, window=window, sinks=2, seed=dim), monkeypatch)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_several_rounds_of_one_row(dim, monkeypatch):
    """The host knows a single row's items: it leaves the join out where none is cut."""
    for new, heads, kv_heads in ((2500, 32, 2), (2432, 16, 16), (2432, 8, 4)):
        check(Step([(new, new + 100)], heads=heads, kv_heads=kv_heads, dim=dim, page=128, seed=new), monkeypatch)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_more_prompts_than_lanes(dim, monkeypatch):
    rng = random.Random(dim)
    same = [(70, 70 + rng.randint(0, 200)) for _ in range(45)]
    check(Step(same, heads=4, kv_heads=4, dim=dim, page=32, seed=dim), monkeypatch)
    ragged = [(n, n + rng.randint(0, 300)) for n in (rng.choice([0, 1, 1, 3, 40, 90, 200]) for _ in range(101))]
    check(Step(ragged, heads=4, kv_heads=2, dim=dim, page=32, seed=dim + 1), monkeypatch)
    check(Step(ragged, heads=6, kv_heads=2, dim=dim, page=16, window=40, sinks=5, seed=dim + 2), monkeypatch)


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (256, BF16), (96, BF16), (64, F32), (256, F32), (48, F32)])
@pytest.mark.parametrize("count", [385, 1000])
def test_more_rows_than_threads(dim, dtype, count, monkeypatch):
    rng = random.Random(count)
    rows = [(rng.choice([0, 1, 1, 1]), rng.choice([1, 16, 33, rng.randint(1, 200)])) for _ in range(count)]
    check(Step(rows, heads=4, kv_heads=2, dim=dim, page=16, dtype=dtype, seed=count), monkeypatch)


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (256, BF16), (64, F32)])
def test_many_verify_rows(dim, dtype, monkeypatch):
    rng = random.Random(dim)
    rows = [(rng.randint(0, 5), rng.randint(5, 300)) for _ in range(700)]
    check(Step(rows, heads=4, kv_heads=1, dim=dim, page=32, dtype=dtype, window=100, sinks=3, seed=dim), monkeypatch)


@pytest.mark.parametrize("dim,dtype", [(96, BF16), (64, F32), (128, F32)])
def test_long_rows_on_the_cuda_cores(dim, dtype, monkeypatch):
    check(Step([(700, 900), (1, 3000), (33, 33)], heads=8, kv_heads=2, dim=dim, page=32, dtype=dtype, seed=dim), monkeypatch)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [[(1, 300), (1, 1), (140, 200), (1, 64)], [(1, 300), (1, 1), (140, 200), (1, 64), (1, 513)],
                                  [(1, 300), (1, 1), (140, 200), (140, 141), (65, 64 + 65)],
                                  [(n, n + 7 * n % 90) for n in range(40, 160, 7)]], ids=["4", "5", "half", "long"])
def test_short_rows_beside_long_ones(dim, rows, monkeypatch):
    """Calls on both sides of the rule that sends short rows another way."""
    check(Step(rows, heads=8, kv_heads=2, dim=dim, page=32, seed=dim, fused=True), monkeypatch)
    check(Step(rows, heads=3, kv_heads=3, dim=dim, page=16, window=60, sinks=2, seed=dim + 1), monkeypatch)
