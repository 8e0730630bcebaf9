"""Infinities and NaN in keys and values behind a window's edge: queries that do not see them give what they give
without them, whichever kernel takes the call, and so do rows of the same call whose caches do not hold them."""
import pytest
import torch

from tests import kv_reference as ref
from tests.test_gpu_attention import BF16, F32, Step

pytestmark = pytest.mark.gpu

WINDOW, SINKS = 50, 3
DECODE, VERIFY = [(1, 200), (1, 61), (1, 1000)], [(4, 300), (7, 90), (5, 64)]
PROMPT = [(200, 450), (90, 90), (150, 777)]
MIXED = [(1, 200), (140, 333), (1, 75), (4, 90), (1, 64), (0, 9)]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rows", [DECODE, VERIFY, PROMPT, MIXED], ids=["decode", "verify", "prompt", "mixed"])
@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (256, BF16), (96, BF16), (64, F32), (256, F32)])
def test_values_behind_a_window(dim, dtype, rows, value):
    s = Step(rows, heads=4, kv_heads=2, dim=dim, dtype=dtype, page=16, window=WINDOW, sinks=SINKS, seed=dim)
    out, spread, logits = s.expected()
    clean = []
    for n, (new, kv) in enumerate(rows[:-1]):  # (the last row's cache stays as it is)
        first = kv - new
        some = [first - WINDOW - 1, first - WINDOW, SINKS if SINKS <= first - WINDOW else -1]  # that no query sees,
        if new > 1:
            some += [first - WINDOW + 1, kv - 1]                                               # that the first, the last
        if new > 20:
            some += [first + new // 2 - WINDOW // 2]                                           # and those between see
        bad = {p for p in some if SINKS <= p < kv}
        for p in bad:
            page = int(s.table[s.table_rows[n]][p // s.page])
            s.kv[0][page, :, p % s.page] = value
            s.kv[1][page, :, p % s.page] = value
        for t in range(new):
            at = first + t
            if not any(at - WINDOW < p <= at for p in bad):
                clean.append(s.token[s.starts[n] + t])
    clean += [s.token[s.starts[-2] + t] for t in range(rows[-1][0])]
    assert len(clean) >= sum(min(new, max(new - 2 - WINDOW, 1)) for new, _ in rows[:-1])
    got, status = s.run()
    tokens = s.max_q * 2
    tol = ref.attention_tolerance(out, spread, logits, max(kv for _, kv in rows), dim, dtype,
                                  24 if dtype == F32 else 8 if tokens > 64 else 16)
    assert status == 0
    assert torch.all((got.double() - out).abs()[clean] <= tol[clean])
    if value != value:
        others = [g for g in s.token if g not in clean]
        assert torch.isnan(got[others].float()).all()
